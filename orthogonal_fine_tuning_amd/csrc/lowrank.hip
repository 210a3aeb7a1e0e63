// Low-rank updates of many requests beside a shared projection, and their
// gradients (oft_lowrank_fwd / oft_lowrank_bwd in oft.h).
//
//   forward   v = x A^T,  y = y_base + scale v B^T
//   backward  u = dy B,   dx = dx_base + scale u A,
//             dA = scale sum_rows u^T x,  dB = scale sum_rows dy^T v
// with the row's own A, B and scale; the segments of a fused projection have
// their own r rows of A and their own columns of v.  All four products with
// rows of activations are two kernels: `down` (activations -> rank, the
// contraction long) and `up` (rank -> activations, the contraction short); the
// backward runs them with the factors' other side along the contraction, read
// with the transposing LDS load.  `pieces` forms the sums over rows.
// Everything is bound by the bytes of x, y, dy and dx, so the products take
// whatever keeps those moving: 16 x 16 x 32 matrix steps (ranks and tiles of
// single decoded rows are small), operands straight from global memory where
// both run along the contraction.
//
// Precision: bf16 factors and activations are matrix operands as they are.
// fp32 values (v, u, fp32 activations) are split into three bf16 parts whose
// sum is the value (split_bf16), whatever the type of the result: where an
// update cancels its base, a bf16 result has as many bits as v does.
#include "adapter_device.h"
#include "gemm_nn.h"
#include "oft_prof.h"

namespace oft {
namespace {

// ------------------------------------------------------------------- down
// v[row][j] = sum_k src[row][k] W[j][k]: a workgroup per 16 XT rows and up to 64
// output columns of one segment (of all, where the rows of src are whole).
// Its DW waves deal the columns of src among them, 64 at a time, so that a long
// contraction is as many loads in flight and no second launch has to add
// partial sums; the waves' sums are added through LDS in their order.  A
// wave's step goes through its own part of LDS, from loads whose lanes run
// along the rows to operands whose lanes run across them.
//
// What `up` takes is written as the operands of its matrix steps, in VP parts
// of bf16, so that it is split once and not by every block of columns: for each
// 16 rows (in list order), each VR columns of v and each 32 of those, a 1 KB
// block a part, lane l's eight items of row l % 16 and columns 8 (l / 16) ...
constexpr int VP = 3;
struct DownArgs {
  RowLists l;
  RowOrder rows;
  const void* src;
  long lds;
  const uint16_t* w;  // a segment's W [r][len], or its transpose [len][r]
  long w_a;           // elements of an adapter's matrices
  float* v;          // [T][R] (NULL: not wanted)
  uint16_t* parts;   // the operands of `up` (NULL: not wanted)
  int vr;            // columns of v that one product of `up` takes
  int R;             // columns of v
  int r, per;        // r output columns a segment (R when whole), `per` a job
  int jobs_per_seg, jobs;
  bool whole;
  int K;
  int seg_at[MAX_SEG + 1];
};

// LIST: LIST_16, or LIST_64 in 4 / XT parts; WT: W is stored transposed
template <int LIST, int XT, int DW, int NG, bool F32, bool WT>
__global__ __launch_bounds__(64 * DW) void down_kernel(DownArgs a) {
  constexpr int P = Oct<F32>::P, SUB = LIST == LIST_16 ? 1 : 4 / XT, ROWS = 16 * XT;
  constexpr int XB = F32 ? 256 : 128, XI = ROWS * XB / 1024;  // bytes of a row of x and step, loads of a lane
  constexpr int WROW = 32 * NG + 16;                        // LDS row of a transposed step: 16 bytes apart in banks
  constexpr int WAVE = ROWS * XB + (WT ? 64 * WROW : 16 * NG * 128);  // bytes of a wave's step
  static_assert(XT == 1 || (!F32 && LIST == LIST_64), "rows of a tile");
  static_assert(DW * WAVE >= DW * XT * NG * 1024, "the sums take the steps' place");
  __shared__ __attribute__((aligned(16))) char lds[DW * WAVE];
  // Tiles in runs to the eight XCDs (workgroup b runs on XCD b % 8): the
  // workgroups that share an L2 read few adapters' W.  (8192 rows of 16
  // adapters, K 2560, 64 columns of v: 18 us, 20 with tile b on workgroup b.)
  int4 e;
  const int tiles = min(a.rows.tiles[LIST], a.l.cap(LIST)) * SUB, total = tiles * a.jobs;
  if ((int)blockIdx.x >= total) return;
  const int xcd = blockIdx.x & 7;
  const int at = xcd * (total >> 3) + min(xcd, total & 7) + (int)(blockIdx.x >> 3);
  const int job = at % a.jobs, tile = at / a.jobs;
  if (!list_entry(a.l, a.rows.tiles, LIST, tile / SUB, e)) return;
  e.y += ROWS * (tile % SUB);
  e.z -= ROWS * (tile % SUB);
  if (e.z <= 0) return;
  e.z = min(e.z, ROWS);
  int seg = 0, col0 = 0, len = a.K;
  if (!a.whole) {
    seg = job / a.jobs_per_seg;
    col0 = a.seg_at[seg];
    len = a.seg_at[seg + 1] - col0;
  }
  const int jw = (job % a.jobs_per_seg) * a.per, nj = min(a.per, a.r - jw);  // rows of the segment's matrix
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l16 = lane & 15, g = lane >> 4;

  if (e.x >= 0) {
    const uint16_t* w = a.w + (size_t)e.x * a.w_a + (size_t)a.r * col0 + (WT ? (size_t)jw : (size_t)jw * len);
    constexpr int XL = XB / 16;  // lanes along a row of x
    size_t xat[XI];
#pragma unroll
    for (int i = 0; i < XI; ++i)
      xat[i] = (size_t)row_at(a.l, a.rows.order, e.y + min(i * (64 / XL) + lane / XL, e.z - 1)) * a.lds + col0 +
               (F32 ? 4 : 8) * (lane % XL);
    size_t wat[2 * NG];
#pragma unroll
    for (int i = 0; i < 2 * NG; ++i) {
      const int t = 64 * i + lane;  // WT: 16 bytes t % 2NG of row t / 2NG of the step
      wat[i] = WT ? (size_t)(t / (2 * NG)) * a.r + 8 * (t % (2 * NG))
                  : (size_t)min(8 * i + (lane >> 3), nj - 1) * len + 8 * (lane & 7);
    }
    const int xk = (F32 ? 4 : 8) * (lane % XL), wk = 8 * (lane & 7);
    char* xs = lds + wave * WAVE;
    char* ws = xs + ROWS * XB;
    // chunks of a row exchanged as in WaveTile, over the 256 bytes of two rows
    // of bf16 or one of fp32
    auto xput = [&](int i) {
      const int r = i * (64 / XL) + lane / XL, c = lane % XL;
      return reinterpret_cast<uint4*>(xs + r * XB + 16 * (F32 ? c ^ r : c ^ ((r >> 1) & 7)));
    };
    auto wput = [&](int r, int c) { return reinterpret_cast<uint4*>(ws + r * 128 + 16 * (c ^ ((r >> 1) & 7))); };

    f32x4 acc[XT][NG];
#pragma unroll
    for (int i = 0; i < XT; ++i)
#pragma unroll
      for (int j = 0; j < NG; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    uint4 x[XI], wv[2 * NG];
    // (segments are multiples of 16: a lane's columns are inside or not)
    auto load = [&](int s) {
      const int k = 64 * s;
#pragma unroll
      for (int i = 0; i < XI; ++i)
        x[i] = k + xk < len ? *reinterpret_cast<const uint4*>(static_cast<const char*>(a.src) + (xat[i] + k) * (F32 ? 4 : 2))
                            : zero4();
#pragma unroll
      for (int i = 0; i < 2 * NG; ++i) {
        const int t = 64 * i + lane;
        if constexpr (WT)
          wv[i] = k + t / (2 * NG) < len && 8 * (t % (2 * NG)) < nj
                      ? *reinterpret_cast<const uint4*>(w + wat[i] + (size_t)k * a.r)
                      : zero4();
        else wv[i] = k + wk < len ? *reinterpret_cast<const uint4*>(w + wat[i] + k) : zero4();
      }
    };
    const int steps = (len + 63) / 64;
    int s = wave;
    if (s < steps) load(s);
    for (; s < steps; s += DW) {  // (a fetch of two steps ahead was no faster)
      wave_order();  // the last step's reads are before these writes
#pragma unroll
      for (int i = 0; i < XI; ++i) *xput(i) = x[i];
#pragma unroll
      for (int i = 0; i < 2 * NG; ++i) {
        const int t = 64 * i + lane;
        if constexpr (WT) *reinterpret_cast<uint4*>(ws + (t / (2 * NG)) * WROW + 16 * (t % (2 * NG))) = wv[i];
        else *wput(8 * i + (lane >> 3), lane & 7) = wv[i];
      }
      if (s + DW < steps) load(s + DW);
      wave_order();
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        uint4 xp[XT][P];
#pragma unroll
        for (int i = 0; i < XT; ++i) {
          const char* row = xs + (16 * i + l16) * XB;
          Oct<F32> o;
          if constexpr (F32) {
            o.a = *reinterpret_cast<const float4*>(row + 16 * ((8 * t + 2 * g) ^ l16));
            o.b = *reinterpret_cast<const float4*>(row + 16 * ((8 * t + 2 * g + 1) ^ l16));
          } else {
            o.u = *reinterpret_cast<const uint4*>(row + 16 * ((4 * t + g) ^ ((l16 >> 1) & 7)));
          }
          o.parts(xp[i]);
        }
#pragma unroll
        for (int j = 0; j < NG; ++j) {
          bf16x8 wj;
          if constexpr (WT) {  // eight rows of column l16 of 16
            const uint16_t* q = reinterpret_cast<const uint16_t*>(ws + (32 * t + 8 * g + (l16 >> 2)) * WROW + 32 * j +
                                                                  8 * (l16 & 3));
            const uint2 lo = nn::ds_read_tr16(q), hi = nn::ds_read_tr16(q + 4 * WROW / 2);
            wj = as_bf16x8(make_uint4(lo.x, lo.y, hi.x, hi.y));
          } else {
            wj = as_bf16x8(*wput(16 * j + l16, 4 * t + g));
          }
#pragma unroll
          for (int i = 0; i < XT; ++i)
#pragma unroll
            for (int p = P - 1; p >= 0; --p) acc[i][j] = mfma16(wj, as_bf16x8(xp[i][p]), acc[i][j]);
        }
      }
    }
    __syncthreads();  // the sums take the steps' place
    float4* red = reinterpret_cast<float4*>(lds);  // [wave][XT NG][64]
#pragma unroll
    for (int i = 0; i < XT; ++i)
#pragma unroll
      for (int j = 0; j < NG; ++j)
        red[((wave * XT + i) * NG + j) * 64 + lane] = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
    __syncthreads();
  }
  // lane: row l16 of 16, four consecutive output columns of 16; rows without
  // an adapter have v = 0
  for (int it = wave; it < XT * NG; it += DW) {
    const int i = it / NG, c0 = 16 * (it % NG) + 4 * g, r = 16 * i + l16;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    if (e.x >= 0) {
      const float4* red = reinterpret_cast<const float4*>(lds);
#pragma unroll
      for (int k = 0; k < DW; ++k) {
        const float4 t = red[(k * XT * NG + it) * 64 + lane];
        o.x += t.x;
        o.y += t.y;
        o.z += t.z;
        o.w += t.w;
      }
    }
    if (c0 >= nj) continue;  // (ranks are multiples of 8)
    const int col = seg * a.r + jw + c0;
    if (a.v != nullptr && r < e.z)
      *reinterpret_cast<float4*>(a.v + (size_t)row_at(a.l, a.rows.order, e.y + r) * a.R + col) = o;
    if (a.parts != nullptr && e.x >= 0 && r < e.z) {
      const int s = col / a.vr, k = col % a.vr, steps = (a.vr + 31) / 32;
      uint16_t* out = a.parts + ((((size_t)tile * XT + i) * (a.R / a.vr) + s) * steps + k / 32) * VP * 512 +
                      ((k % 32) / 8 * 16 + l16) * 8 + k % 8;
      uint32_t h[4][VP];
      split_bf16<VP>(o.x, h[0]);
      split_bf16<VP>(o.y, h[1]);
      split_bf16<VP>(o.z, h[2]);
      split_bf16<VP>(o.w, h[3]);
#pragma unroll
      for (int p = 0; p < VP; ++p)
        *reinterpret_cast<uint2*>(out + p * 512) = make_uint2(h[0][p] | (h[1][p] << 16), h[2][p] | (h[3][p] << 16));
    }
  }
}

// --------------------------------------------------------------------- up
// out[row][c] = base[row][c] + scale sum_k v[row][k] W[c][k]: a wave per tile
// of rows and 64 columns of one segment, v from the operands that `down` left.
// The columns that a matrix step's operand rows stand for are chosen so that a
// lane's results are the 16 bytes of a row next to its neighbours': bf16
// column 32 (m / 2) + 8 (i / 4) + 4 (m % 2) + i % 4 of the 64 for operand row i
// of step m, fp32 16 m + i.
struct UpArgs {
  RowLists l;
  RowOrder rows;
  const uint16_t* parts;
  int r, segs;        // the contraction, and how many there are in a row of v
  const uint16_t* w;  // [n][C][r], or its transpose [n][r][C]
  long w_a;
  const float* scale;
  const void* base;
  void* out;
  int C;  // columns
  int n_seg, blocks;
  int seg_at[MAX_SEG + 1], block_at[MAX_SEG + 1];  // columns and 64-column blocks before each segment
};
constexpr int UC = 64;

// The wave's 64 columns.
struct UpBlock {
  int seg, n0, hi;
};
__device__ __forceinline__ UpBlock up_block(const UpArgs& a, int cb) {
  UpBlock b{0, UC * cb, a.seg_at[1]};
#pragma unroll
  for (int i = 1; i < MAX_SEG; ++i)
    if (i < a.n_seg && cb >= a.block_at[i]) b = UpBlock{i, a.seg_at[i] + UC * (cb - a.block_at[i]), a.seg_at[i + 1]};
  return b;
}

// W of the wave's columns as operands, contraction items k0 + 32 s .. (zero
// past r): step m's rows are columns as above.  A transposed W comes through
// the wave's tile, 64 items at a time, and the transposing load.
template <bool F32, bool WT>
struct UpOperand {
  const UpArgs& a;
  const uint16_t* w;
  const UpBlock& b;
  WaveTile t;
  int lane;
  __device__ __forceinline__ void stage(int k0) const {
    if constexpr (WT) {
      uint4 u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = k0 + 8 * i + (lane >> 3), c = b.n0 + 8 * (lane & 7);
        u[i] = k < a.r && c < b.hi ? *reinterpret_cast<const uint4*>(w + (size_t)k * a.C + c) : zero4();
      }
      wave_order();
#pragma unroll
      for (int i = 0; i < 8; ++i) t.by_row(i, lane) = u[i];
      wave_order();
    }
  }
  __device__ __forceinline__ void get(int k0, int s, bf16x8 (&o)[4]) const {
    const int l16 = lane & 15, g = lane >> 4;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int first = F32 ? 16 * m : 32 * (m / 2) + 4 * (m % 2);
      constexpr int APART = F32 ? 4 : 8;  // columns between the quarters of an operand's rows
      if constexpr (WT) {
        // the 16-lane group's eight-byte pieces: four columns of row l16 / 4 each
        const int c = first + APART * (l16 & 3), k = 32 * s + 8 * g + (l16 >> 2);
        const uint2 lo = nn::ds_read_tr16(reinterpret_cast<const uint16_t*>(t.at(k, c >> 3)) + (c & 7));
        const uint2 hi = nn::ds_read_tr16(reinterpret_cast<const uint16_t*>(t.at(k + 4, c >> 3)) + (c & 7));
        o[m] = as_bf16x8(make_uint4(lo.x, lo.y, hi.x, hi.y));
      } else {
        const int c = min(b.n0 + first + APART * (l16 >> 2) + (l16 & 3), b.hi - 1), k = k0 + 32 * s + 8 * g;
        o[m] = as_bf16x8(k < a.r ? *reinterpret_cast<const uint4*>(w + (size_t)c * a.r + k) : zero4());
      }
    }
  }
};

// v of 16 rows (block `i16` of the list's, `rows` of them there) and contraction
// items 32 s ..
__device__ __forceinline__ void up_rows(const UpArgs& a, int seg, int i16, int rows, int s, int lane,
                                        bf16x8 (&o)[VP]) {
  const uint16_t* p =
      a.parts + (((size_t)i16 * a.segs + seg) * ((a.r + 31) / 32) + s) * VP * 512 + 8 * lane;
  const bool ok = 32 * s + 8 * (lane >> 4) < a.r && (lane & 15) < rows;  // (nothing else is written)
#pragma unroll
  for (int k = 0; k < VP; ++k) o[k] = as_bf16x8(zero4());
  if (ok) {  // (one branch: a choice per load made the compiler wait between them)
#pragma unroll
    for (int k = 0; k < VP; ++k) o[k] = as_bf16x8(*reinterpret_cast<const uint4*>(p + k * 512));
  }
}

// Decoded rows, and rows of fp32: four waves, base and result by operands.
template <int TM, bool F32, bool WT>
__global__ __launch_bounds__(256) void up_kernel(UpArgs a) {
  constexpr int XG = TM / 16, H = F32 ? 4 : 2;  // H: 16-byte pieces of a lane and row
  __shared__ __attribute__((aligned(16))) char lds[WT ? 4 : 1][WT ? WaveTile::BYTES : 16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  const int wgs = (a.blocks + 3) / 4, tile = blockIdx.x / wgs, cb = (blockIdx.x % wgs) * 4 + wave;
  int4 e;
  if (cb >= a.blocks || !list_entry(a.l, a.rows.tiles, TM == 16 ? LIST_16 : LIST_64, tile, e)) return;
  const UpBlock b = up_block(a, cb);
  const UpOperand<F32, WT> w{a, a.w + (size_t)max(e.x, 0) * a.w_a, b, WaveTile{lds[WT ? wave : 0]}, lane};
  // what does not wait for the rows' numbers first
  bf16x8 wo[4], v[XG][VP];
  auto operands = [&](int k0, int s) {
    w.get(k0, s, wo);
#pragma unroll
    for (int i = 0; i < XG; ++i) up_rows(a, b.seg, tile * XG + i, e.z - 16 * i, k0 / 32 + s, lane, v[i]);
  };
  if (e.x >= 0) {
    w.stage(0);
    operands(0, 0);
  }
  // column of piece h within the 64
  auto col = [&](int h) { return F32 ? 16 * h + 4 * g : 32 * h + 8 * g; };
  uint4 y[XG][H];
  size_t at[XG];
#pragma unroll
  for (int i = 0; i < XG; ++i) {
    at[i] = (size_t)row_at(a.l, a.rows.order, e.y + min(16 * i + l16, e.z - 1)) * a.C + b.n0;
#pragma unroll
    for (int h = 0; h < H; ++h) {
      // (segments are multiples of 16: a piece is inside or not)
      const bool ok = b.n0 + col(h) < b.hi && a.base != nullptr;
      y[i][h] = ok ? *reinterpret_cast<const uint4*>(static_cast<const char*>(a.base) + (at[i] + col(h)) * (F32 ? 4 : 2))
                   : zero4();
    }
  }
  auto store = [&](int i, int h, const uint4& u) {
    if (16 * i + l16 < e.z && b.n0 + col(h) < b.hi)
      *reinterpret_cast<uint4*>(static_cast<char*>(a.out) + (at[i] + col(h)) * (F32 ? 4 : 2)) = u;
  };
  if (e.x < 0) {  // rows of the base model
    if (a.base == a.out) return;
#pragma unroll
    for (int i = 0; i < XG; ++i)
#pragma unroll
      for (int h = 0; h < H; ++h) store(i, h, y[i][h]);
    return;
  }
  const float sc = a.scale[e.x];
  f32x4 acc[XG][4];
#pragma unroll
  for (int i = 0; i < XG; ++i)
#pragma unroll
    for (int m = 0; m < 4; ++m) acc[i][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < a.r; k += 32) {
    if (k > 0) {
      if (k % 64 == 0) w.stage(k);
      operands(k & ~63, k / 32 % 2);
    }
#pragma unroll
    for (int i = 0; i < XG; ++i)
#pragma unroll
      for (int p = VP - 1; p >= 0; --p)
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[i][m] = mfma16(wo[m], v[i][p], acc[i][m]);
  }
#pragma unroll
  for (int i = 0; i < XG; ++i)
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const uint32_t u[4] = {y[i][h].x, y[i][h].y, y[i][h].z, y[i][h].w};
      uint32_t q[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if constexpr (F32) {
          q[c] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, u[c]) + sc * acc[i][h][c]);
        } else {
          const f32x4& s = acc[i][2 * h + c / 2];
          q[c] = pack_bf16x2(bf16_to_f32(u[c] & 0xFFFF) + sc * s[2 * (c % 2)],
                             bf16_to_f32(u[c] >> 16) + sc * s[2 * (c % 2) + 1]);
        }
      }
      store(i, h, make_uint4(q[0], q[1], q[2], q[3]));
    }
}

// bf16 rows in tiles of 64: base and result go through the wave's tile, so
// that they are read and written by whole stretches of rows.  KS: 32-item
// steps of the contraction whose W the wave keeps in registers while it takes
// its rows 16 at a time; 0: any number, all rows at once.
constexpr int UW = 2;  // waves of a workgroup; they share nothing

template <bool STREAM, bool WT, int KS>
__global__ __launch_bounds__(64 * UW) void up_tile_kernel(UpArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[UW][WaveTile::BYTES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4;
  const int wgs = (a.blocks + UW - 1) / UW, tile = blockIdx.x / wgs, cb = (blockIdx.x % wgs) * UW + wave;
  int4 e;
  if (cb >= a.blocks || !list_entry(a.l, a.rows.tiles, LIST_64, tile, e)) return;
  const UpBlock b = up_block(a, cb);
  const int c = b.n0 + 8 * (lane & 7);  // (segments are multiples of 16: a piece is inside or not)
  const WaveTile t{lds[wave]};
  int row[8];
  tile_rows8(a.l, a.rows.order, e, lane, row);
  Oct<false> y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c < b.hi && a.base != nullptr) y[i].load<STREAM>(a.base, (size_t)row[i] * a.C + c);
    else y[i].zero();
  if (e.x >= 0) {
    const UpOperand<false, WT> w{a, a.w + (size_t)e.x * a.w_a, b, t, lane};
    const float sc = a.scale[e.x];
    // 16 rows' results onto their base in the tile
    auto add = [&](int i, const f32x4 (&acc)[4]) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4& at = t.by_operand(i, 4 * h + g, lane);
        const uint4 o = at;
        const uint32_t u[4] = {o.x, o.y, o.z, o.w};
        uint32_t q[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const f32x4& s = acc[2 * h + k / 2];
          q[k] = pack_bf16x2(bf16_to_f32(u[k] & 0xFFFF) + sc * s[2 * (k % 2)],
                             bf16_to_f32(u[k] >> 16) + sc * s[2 * (k % 2) + 1]);
        }
        at = make_uint4(q[0], q[1], q[2], q[3]);
      }
    };
    auto fill = [&]() {
      wave_order();
#pragma unroll
      for (int i = 0; i < 8; ++i) t.by_row(i, lane) = y[i].u;
      wave_order();
    };
    if constexpr (KS > 0) {
      // v of 16 rows is fetched while the 16 before are multiplied
      bf16x8 wo[KS][4], v[2][KS][VP];
      auto fetch = [&](int i) {
#pragma unroll
        for (int s = 0; s < KS; ++s) up_rows(a, b.seg, 4 * tile + i, e.z - 16 * i, s, lane, v[i % 2][s]);
      };
      fetch(0);
      w.stage(0);
#pragma unroll
      for (int s = 0; s < KS; ++s) w.get(0, s, wo[s]);
      fill();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < 3) fetch(i + 1);
        f32x4 acc[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int p = VP - 1; p >= 0; --p)
#pragma unroll
            for (int m = 0; m < 4; ++m) acc[m] = mfma16(wo[s][m], v[i % 2][s][p], acc[m]);
        add(i, acc);
      }
    } else {
      f32x4 acc[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int m = 0; m < 4; ++m) acc[i][m] = f32x4{0.f, 0.f, 0.f, 0.f};
      for (int k0 = 0; k0 < a.r; k0 += 64) {
        w.stage(k0);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (k0 + 32 * s >= a.r) break;
          bf16x8 wo[4];
          w.get(k0, s, wo);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            bf16x8 v[VP];
            up_rows(a, b.seg, 4 * tile + i, e.z - 16 * i, k0 / 32 + s, lane, v);
#pragma unroll
            for (int p = VP - 1; p >= 0; --p)
#pragma unroll
              for (int m = 0; m < 4; ++m) acc[i][m] = mfma16(wo[m], v[p], acc[i][m]);
          }
        }
      }
      fill();
#pragma unroll
      for (int i = 0; i < 4; ++i) add(i, acc[i]);
    }
    wave_order();
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i].u = t.by_row(i, lane);
  } else if (a.base == a.out) {
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (8 * i + (lane >> 3) < e.z && c < b.hi) y[i].store<STREAM>(a.out, (size_t)row[i] * a.C + c);
}

// ------------------------------------------------------------------ pieces
// Sums over an adapter's rows: out[j][c] = scale sum_rows U[row][j] X[row][c]
// for 256 columns of X and up to 32 of U, over one piece of the adapter's
// rows.  Both operands run along the rows here: tiles of PR rows go to LDS in
// row order and are read with the transposing LDS load.  U is fp32 in three
// parts; so is X where it is fp32.  A second part is below 2^-7 of the value, a
// third below 2^-15: the product of the two third parts, below 2^-30, is left
// out, all others are taken (777 rows of rank 24 beside QKV 18.4 us, 18.0
// without those of a second and a third part, 8192 of rank 32 on gate/up 148
// and 144).  A step's rows are fetched two steps ahead.
constexpr int PC = 256;
constexpr int MAXG = 2;               // 16-column groups of U a workgroup: more keep a CU to three workgroups
constexpr int LDX = PC + 16;  // LDS row: 16 elements more, so that the four rows of a transposing read lie in different banks

struct PieceJob {
  const void* x;
  long ldx;
  const float* u;
  float* out;      // [n][...], element (j, c) at j so_j + c so_c
  long out_a;
  long part_off;   // this sum's place in a partial slot
  int so_j, so_c;
  int blocks;      // column blocks, over all segments
  int nj, njc;     // columns of U a segment, and the jobs they are cut into
  int n_seg;
  bool whole;      // one segment of all columns
  int seg_at[MAX_SEG + 1], block_at[MAX_SEG + 1];
};
struct PieceArgs {
  RowLists l;
  RowOrder rows;
  int list, R;
  const float* scale;
  float* part;
  long slot;  // floats of a partial slot
};

template <int NJ, int PR, bool F32>
__device__ __forceinline__ void piece(const PieceArgs& a, const PieceJob& q, int4 e, int job, uint16_t* xs, uint16_t* us,
                                      int* idx) {
  constexpr int PX = Oct<F32>::P, LDU = NJ * 16 + 16;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  const int cb = job / q.njc, jc = job % q.njc;
  int seg = 0, c_lo = q.seg_at[0], c_hi = q.seg_at[1], b_lo = 0;
#pragma unroll
  for (int i = 1; i < MAX_SEG; ++i)
    if (i < q.n_seg && cb >= q.block_at[i]) {
      seg = i;
      c_lo = q.seg_at[i];
      c_hi = q.seg_at[i + 1];
      b_lo = q.block_at[i];
    }
  const int c0 = c_lo + PC * (cb - b_lo);
  const int j0 = NJ * 16 * jc, nj = min(NJ * 16, q.nj - j0);
  const int ju = (q.whole ? 0 : seg * q.nj) + j0;  // column of U

  f32x4 acc[NJ][4];  // of the rows whose numbers are in LDS
  // thread: 8 columns of rows tid / 32 + 8 i of a step; U: 4 columns of rows
  // tid / UT + UR i
  constexpr int XI = PR / 8;
  const int xc = c0 + 8 * (tid & 31), xr = tid >> 5;
  const bool xok = xc < c_hi;
  constexpr int UT = 4 * NJ, UR = 256 / UT, UI = (PR + UR - 1) / UR;
  const int uc = 4 * (tid % UT), ur = tid / UT;
  const bool uok = ur < UR && uc < nj;
  struct Tile {
    Oct<F32> x[XI];
    float4 u[UI];
  } even, odd;
  // rows r0 .. of the `rows` whose numbers are in LDS
  auto load = [&](int r0, int rows, Tile& t) {
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      const int r = r0 + xr + 8 * i;
      if (r < rows && xok) t.x[i].load(q.x, (size_t)idx[r] * q.ldx + xc);
      else t.x[i].zero();
    }
#pragma unroll
    for (int i = 0; i < UI; ++i) {
      const int r = r0 + ur + UR * i;
      t.u[i] = r < rows && uok ? *reinterpret_cast<const float4*>(q.u + (size_t)idx[r] * a.R + ju + uc)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  auto step = [&](int r0, int rows, Tile& t) {
    __syncthreads();  // the last step's reads are done
#pragma unroll
    for (int i = 0; i < XI; ++i) {
      uint4 p[PX];
      t.x[i].parts(p);
#pragma unroll
      for (int k = 0; k < PX; ++k)
        *reinterpret_cast<uint4*>(xs + (k * PR + xr + 8 * i) * LDX + 8 * (tid & 31)) = p[k];
    }
#pragma unroll
    for (int i = 0; i < UI; ++i)
      if (ur < UR && ur + UR * i < PR) {
        const float v[4] = {t.u[i].x, t.u[i].y, t.u[i].z, t.u[i].w};
        uint32_t h[4][3];
#pragma unroll
        for (int k = 0; k < 4; ++k) split_bf16<3>(v[k], h[k]);
#pragma unroll
        for (int p = 0; p < 3; ++p)
          *reinterpret_cast<uint2*>(us + (p * PR + ur + UR * i) * LDU + uc) =
              make_uint2(h[0][p] | (h[1][p] << 16), h[2][p] | (h[3][p] << 16));
      }
    if (r0 + 2 * PR < rows) load(r0 + 2 * PR, rows, t);
    __syncthreads();
#pragma unroll
    for (int k0 = 0; k0 < PR; k0 += 32) {
      // lane l16 of group g: rows 8 g .. 8 g + 7 of column l16 of 16
      const int tr = k0 + 8 * g + (l16 >> 2), tc = 4 * (l16 & 3);
      bf16x8 xv[4][PX];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int k = 0; k < PX; ++k) {
          const uint16_t* p = xs + (k * PR + tr) * LDX + 64 * wave + 16 * c + tc;
          const uint2 lo = nn::ds_read_tr16(p), hi = nn::ds_read_tr16(p + 4 * LDX);
          xv[c][k] = as_bf16x8(make_uint4(lo.x, lo.y, hi.x, hi.y));
        }
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int p = 2; p >= 0; --p) {
          const uint16_t* s = us + (p * PR + tr) * LDU + 16 * j + tc;
          const uint2 lo = nn::ds_read_tr16(s), hi = nn::ds_read_tr16(s + 4 * LDU);
          const bf16x8 uv = as_bf16x8(make_uint4(lo.x, lo.y, hi.x, hi.y));
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int k = PX - 1; k >= 0; --k)
              if (p + k <= 3) acc[j][c] = mfma16(uv, xv[c][k], acc[j][c]);
        }
    }
  };
  // lane: column l16 of 16, rows (of U^T) 4 g .. 4 g + 3 of 16.  The sums of
  // further rows are added to those that the lane wrote itself.
  const float sc = a.scale[e.x];
  float* out = e.w < 0 ? q.out + (size_t)e.x * q.out_a : a.part + (size_t)e.w * a.slot + q.part_off;
  auto write = [&](bool first) {
    int col0 = c0 + 64 * wave + l16;  // (opaque: the addresses are not kept in registers over the rows)
    asm volatile("" : "+v"(col0));
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int jj = 16 * j + 4 * g;
      if (jj >= nj) continue;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int col = col0 + 16 * c;
        if (col >= c_hi) continue;
        float* o = out + (size_t)(j0 + jj) * q.so_j + (size_t)col * q.so_c;
        f32x4 v = sc * acc[j][c];
        if (q.so_j == 1) {
          if (!first) v += *reinterpret_cast<const f32x4*>(o);
          *reinterpret_cast<f32x4*>(o) = v;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) o[(size_t)k * q.so_j] = first ? v[k] : o[(size_t)k * q.so_j] + v[k];
        }
      }
    }
  };
  for (int from = 0; from < e.z; from += IDX) {
    const int rows = min(IDX, e.z - from);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[j][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    __syncthreads();
    fetch_rows(a.l, a.rows.order, e.y + from, rows, idx);
    __syncthreads();
    load(0, rows, even);
    load(PR, rows, odd);
    for (int r0 = 0; r0 < rows; r0 += 2 * PR) {
      step(r0, rows, even);
      if (r0 + PR < rows) step(r0 + PR, rows, odd);
    }
    write(from == 0);
  }
}

template <int NA, int NB, bool F32>
__global__ __launch_bounds__(256, F32 ? 2 : 4) void piece_kernel(PieceArgs a, PieceJob qa, PieceJob qb) {
  constexpr int NJ = NA > NB ? NA : NB, PR = 32;
  __shared__ __attribute__((aligned(16))) uint16_t xs[Oct<F32>::P * PR * LDX];
  __shared__ __attribute__((aligned(16))) uint16_t us[3 * PR * (NJ * 16 + 16)];
  __shared__ int idx[IDX];
  int4 e;
  if (!list_entry(a.l, a.rows.tiles, a.list, blockIdx.y, e) || e.x < 0) return;
  e.w = min(e.w, RowLists::slots(a.list) - 1);
  const int ja = qa.blocks * qa.njc;
  if ((int)blockIdx.x < ja) piece<NA, PR, F32>(a, qa, e, blockIdx.x, xs, us, idx);
  else piece<NB, PR, false>(a, qb, e, blockIdx.x - ja, xs, us, idx);
}

// The pieces of an adapter of two or more, in order; zeros for an adapter
// without rows.  (An adapter of one piece has its result already.)
struct JoinArgs {
  RowLists l;
  const int* offsets;
  const int* tiles;
  int list;
  const float* part;
  long slot, off[2], per[2];  // the two sums' places in a slot, and sizes
  float* out[2];
};
__global__ __launch_bounds__(256) void join_kernel(JoinArgs a) {
  const int ad = blockIdx.y;
  const int pieces = a.l.count(a.list, a.offsets[ad + 1] - a.offsets[ad]);
  if (pieces == 1) return;
  int first;
  const int slots = slots_of(a.l, a.tiles, a.list, ad, pieces, first);
  long i = 4 * ((long)blockIdx.x * 256 + threadIdx.x);
  int which = 0;
  if (i >= a.per[0]) {
    i -= a.per[0];
    which = 1;
  }
  if (i >= a.per[which]) return;
  const float* p = a.part + (size_t)first * a.slot + a.off[which] + i;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < slots; ++k, p += a.slot) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  }
  *reinterpret_cast<float4*>(a.out[which] + (size_t)ad * a.per[which] + i) = s;
}

// ------------------------------------------------------------------- plans
size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

// Rows of a tile: 16 while the batch is one of decoded rows (an adapter then
// has few), else 64; small ranks gain longer, since the factors that each tile
// reads again are small.  Forward calls in us by 16 and by 64 rows, 8 adapters
// and 64: rank 16 beside QKV, 2048 rows 21.5, 21.9 and 22.5, 29, gradients 43, 42
// and 54, 56; 4096 rows 32, 34 and 34, 36, but the gradients 61, 59 and 76, 76,
// and one rule serves both; rank 64 beside QKV, 512 rows of 4 and 64 adapters
// 17, 17 and 32, 35, gradients of 4 and 16 40, 48 and 52, 59; on gate/up, 256
// rows 20, 21 and 56, 52; 512 rows 27, 27 and 61, 54; 1024 rows 42, 35 and 80, 73.
int tile_rows(int T, int r) { return T <= (r <= 32 ? T16_MAX : 512) ? 16 : 64; }

struct Plan {
  RowLists l;
  int tm, R;
  int list;
  size_t v, parts, sums, bytes;  // workspace: v, its operands for `up`, partial sums of the gradients
  long slot;
};
Plan plan_of(const LowrankDims& d, bool bwd) {
  Plan p;
  p.l = RowLists{d.T, d.n};
  p.tm = tile_rows(d.T, d.r);
  p.R = d.n_seg * d.r;
  p.v = 0;
  p.parts = bwd ? up256(4 * (size_t)d.T * p.R) : 0;
  const size_t tiles16 = p.tm == 16 ? p.l.cap(LIST_16) : 4 * (size_t)p.l.cap(LIST_64);
  const size_t steps = bwd ? (p.R + 31) / 32 : (size_t)d.n_seg * ((d.r + 31) / 32);
  p.bytes = p.parts + tiles16 * steps * VP * 1024;
  p.sums = 0;
  p.slot = (long)p.R * d.K + (long)d.N * d.r;
  p.list = LIST_SHORT;
  if (bwd) {
    p.sums = p.bytes;
    // pieces of a quarter of the rows where the columns alone give workgroups
    // enough, or bf16 rows are few: fewer partial sums (us of a backward pass of
    // one adapter by quarters and by sixteenths, K 2560: rank 64 beside QKV,
    // 108 workgroups a piece, 2048 rows 84 and 94, of fp32 100 and 101; on
    // gate/up, 212 of them, 94 and 117, 120 and 131; rank 16 on gate/up, 86 of
    // them, 56 and 56, 87 and 70; beside QKV, 44 of them, 46 and 43, 71 and 57,
    // but 512 rows of bf16 26 and 27, 1024 rows 32 and 33)
    const auto jobs = [](int cols, int r) { return (cols + PC - 1) / PC * ((r + 16 * MAXG - 1) / (16 * MAXG)); };
    p.list = jobs(d.K, p.R) + jobs(d.N, d.r) >= 100 || (!d.f32 && d.T <= 1024) ? LIST_LONG : LIST_SHORT;
    p.bytes = p.sums + up256(4 * (size_t)RowLists::slots(p.list) * p.slot);
  }
  return p;
}

template <class F>
void groups_of(int ng, F f) {
  switch (ng) {
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    case 3: f(std::integral_constant<int, 3>{}); break;
    default: f(std::integral_constant<int, 4>{}); break;
  }
}

// r output columns for each of n_seg segments (one when whole).  Decoded rows
// (LIST_16) are few and long: 16 columns of v a workgroup, so that more of them
// share A (64 rows, K 2560, 48 columns: 7.0 us, 8.8 with all in one).  Many
// rows: 32 at a time, each of which reads all of W, and four waves; that takes
// 256 workgroups to fill the chip (8192 rows 20 us, 22 by 16 rows and eight
// waves; 2048 rows 13 and 9).
void run_down(const Plan& p, DownArgs a, int n_seg, bool f32, hipStream_t st) {
  const int groups = (a.r + 15) / 16, most = p.tm == 16 ? 1 : 4;
  a.jobs_per_seg = (groups + most - 1) / most;
  const int ng = (groups + a.jobs_per_seg - 1) / a.jobs_per_seg;
  a.per = 16 * ng;
  const int jobs = a.jobs = n_seg * a.jobs_per_seg;
  const bool wide = p.tm != 16 && !(a.whole && f32) && ng >= 2 && (long)(p.l.T / 32) * jobs >= 256;
  auto run = [&](auto list, auto xt, auto dw, auto ng, auto f, auto wt) {
    constexpr int LIST = decltype(list)::value, XT = decltype(xt)::value, DW = decltype(dw)::value;
    const dim3 grid((unsigned)p.l.cap(LIST) * (LIST == LIST_16 ? 1 : 4 / XT) * jobs);
    hipLaunchKernelGGL((down_kernel<LIST, XT, DW, decltype(ng)::value, decltype(f)::value, decltype(wt)::value>), grid,
                       dim3(64 * DW), 0, st, a);
  };
  using std::integral_constant;
  using I1 = integral_constant<int, 1>;
  auto rows = [&](auto f, auto wt) {
    if (p.tm == 16) {
      run(integral_constant<int, LIST_16>{}, I1{}, integral_constant<int, 8>{}, I1{}, f, wt);
      return;
    }
    groups_of(ng, [&](auto c) {
      constexpr int NG = decltype(c)::value;
      const integral_constant<int, LIST_64> list;
      if constexpr (NG >= 2 && !decltype(f)::value) {
        if (wide) {
          run(list, integral_constant<int, 2>{}, integral_constant<int, 4>{}, c, f, wt);
          return;
        }
      }
      run(list, I1{}, integral_constant<int, 8>{}, c, f, wt);
    });
  };
  if (!a.whole) rows(std::false_type{}, std::true_type{});  // (dy is bf16)
  else if (f32) rows(std::true_type{}, std::false_type{});
  else rows(std::false_type{}, std::false_type{});
}

template <bool WT>
void run_up(const Plan& p, UpArgs a, bool f32, hipStream_t st) {
  a.block_at[0] = 0;
  for (int i = 0; i < MAX_SEG; ++i)
    a.block_at[i + 1] = i < a.n_seg ? a.block_at[i] + (a.seg_at[i + 1] - a.seg_at[i] + UC - 1) / UC : a.block_at[i];
  a.blocks = a.block_at[a.n_seg];
  const unsigned tiles = p.l.cap(p.tm == 16 ? LIST_16 : LIST_64);
  const dim3 grid(tiles * ((a.blocks + 3) / 4));
  if (p.tm == 16) {
    if (f32) hipLaunchKernelGGL((up_kernel<16, true, WT>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((up_kernel<16, false, WT>), grid, dim3(256), 0, st, a);
  } else if (f32) {
    hipLaunchKernelGGL((up_kernel<64, true, WT>), grid, dim3(256), 0, st, a);
  } else {
    auto run = [&](auto stream, auto ks) {
      hipLaunchKernelGGL((up_tile_kernel<decltype(stream)::value, WT, decltype(ks)::value>),
                         dim3(tiles * ((a.blocks + UW - 1) / UW)), dim3(64 * UW), 0, st, a);
    };
    auto steps = [&](auto stream) {
      if (a.r <= 32) run(stream, std::integral_constant<int, 1>{});
      else if (a.r <= 64) run(stream, std::integral_constant<int, 2>{});
      else run(stream, std::integral_constant<int, 0>{});
    };
    if ((size_t)p.l.T * a.C * 2 > STREAM_BYTES) steps(std::true_type{});
    else steps(std::false_type{});
  }
}

// columns before each segment
void segments(const LowrankDims& d, int (&at)[MAX_SEG + 1]) {
  at[0] = 0;
  for (int i = 0; i < MAX_SEG; ++i) at[i + 1] = at[i] + (i < d.n_seg ? d.seg[i] : 0);
}
void one_segment(int cols, int (&at)[MAX_SEG + 1]) {
  at[0] = 0;
  for (int i = 1; i <= MAX_SEG; ++i) at[i] = cols;
}

void blocks_of(PieceJob& q, int per) {
  q.block_at[0] = 0;
  for (int i = 0; i < MAX_SEG; ++i)
    q.block_at[i + 1] = i < q.n_seg ? q.block_at[i] + (q.seg_at[i + 1] - q.seg_at[i] + per - 1) / per : q.block_at[i];
  q.blocks = q.block_at[q.n_seg];
}

}  // namespace

size_t lowrank_ws_bytes(const LowrankDims& d, bool bwd) { return plan_of(d, bwd).bytes; }

hipError_t launch_lowrank_fwd(const LowrankDims& d, const LowrankPtrs& q, char* ws, hipStream_t st) {
  ProfScope prof(st, "lowrank.fwd");
  const Plan p = plan_of(d, false);
  uint16_t* parts = reinterpret_cast<uint16_t*>(ws + p.parts);
  DownArgs a{};
  a.l = p.l;
  a.rows = q.rows;
  a.src = q.x;
  a.lds = d.K;
  a.w = q.A;
  a.w_a = (long)p.R * d.K;
  a.v = q.v;
  a.parts = parts;
  a.vr = d.r;
  a.R = p.R;
  a.r = p.R;
  a.whole = true;
  a.K = d.K;
  run_down(p, a, 1, d.f32, st);
  UpArgs b{};
  b.l = p.l;
  b.rows = q.rows;
  b.parts = parts;
  b.r = d.r;
  b.segs = d.n_seg;
  b.w = q.B;
  b.w_a = (long)d.N * d.r;
  b.scale = q.scale;
  b.base = q.y_base;
  b.out = q.y;
  b.C = d.N;
  b.n_seg = d.n_seg;
  segments(d, b.seg_at);
  run_up<false>(p, b, d.f32, st);
  return hipGetLastError();
}

hipError_t launch_lowrank_bwd(const LowrankDims& d, const LowrankGradPtrs& q, char* ws, hipStream_t st) {
  ProfScope prof(st, "lowrank.bwd");
  const Plan p = plan_of(d, true);
  float* u = reinterpret_cast<float*>(ws + p.v);
  uint16_t* parts = reinterpret_cast<uint16_t*>(ws + p.parts);
  float* sums = reinterpret_cast<float*>(ws + p.sums);

  // (without rows only the gradients' zeros are left to write)
  if (d.T > 0 && (q.dx != nullptr || q.dA != nullptr)) {
    DownArgs a{};
    a.l = p.l;
    a.rows = q.rows;
    a.src = q.dy;
    a.lds = d.N;
    a.w = q.B;
    a.w_a = (long)d.N * d.r;
    a.v = q.dA != nullptr ? u : nullptr;
    a.parts = q.dx != nullptr ? parts : nullptr;
    a.vr = p.R;
    a.R = p.R;
    a.r = d.r;
    a.whole = false;
    segments(d, a.seg_at);
    run_down(p, a, d.n_seg, false, st);
  }
  if (d.T > 0 && q.dx != nullptr) {
    UpArgs b{};
    b.l = p.l;
    b.rows = q.rows;
    b.parts = parts;
    b.r = p.R;
    b.segs = 1;
    b.w = q.A;
    b.w_a = (long)p.R * d.K;
    b.scale = q.scale;
    b.base = q.dx_base;
    b.out = q.dx;
    b.C = d.K;
    b.n_seg = 1;
    one_segment(d.K, b.seg_at);
    run_up<true>(p, b, d.f32, st);
  }
  if (q.dA == nullptr && q.dB == nullptr) return hipGetLastError();

  PieceArgs a{};
  a.l = p.l;
  a.rows = q.rows;
  a.list = p.list;
  a.R = p.R;
  a.scale = q.scale;
  a.part = sums;
  a.slot = p.slot;
  PieceJob ja{}, jb{};
  ja.x = q.x;
  ja.ldx = d.K;
  ja.u = u;
  ja.out = q.dA;
  ja.out_a = (long)p.R * d.K;
  ja.part_off = 0;
  ja.so_j = d.K;
  ja.so_c = 1;
  ja.n_seg = 1;
  ja.whole = true;
  ja.nj = p.R;
  one_segment(d.K, ja.seg_at);
  blocks_of(ja, PC);
  jb.x = q.dy;
  jb.ldx = d.N;
  jb.u = q.v;
  jb.out = q.dB;
  jb.out_a = (long)d.N * d.r;
  jb.part_off = (long)p.R * d.K;
  jb.so_j = 1;
  jb.so_c = d.r;
  jb.n_seg = d.n_seg;
  jb.nj = d.r;
  segments(d, jb.seg_at);
  blocks_of(jb, PC);
  // columns of U a workgroup takes: up to 16 MAXG, evenly
  const int ga = (p.R + 15) / 16, gb = (d.r + 15) / 16;
  ja.njc = (ga + MAXG - 1) / MAXG;
  jb.njc = (gb + MAXG - 1) / MAXG;
  const int na = (ga + ja.njc - 1) / ja.njc, nb = (gb + jb.njc - 1) / jb.njc;
  if (q.dA == nullptr) ja.blocks = 0;
  if (q.dB == nullptr) jb.blocks = 0;
  const dim3 grid(ja.blocks * ja.njc + jb.blocks * jb.njc, p.l.cap(p.list));
  auto pairs_of = [](int g, auto f) { g == 1 ? f(std::integral_constant<int, 1>{}) : f(std::integral_constant<int, MAXG>{}); };
  if (d.T > 0) pairs_of(na, [&](auto va) {
    pairs_of(nb, [&](auto vb) {
      constexpr int NA = decltype(va)::value, NB = decltype(vb)::value;
      if (d.f32) hipLaunchKernelGGL((piece_kernel<NA, NB, true>), grid, dim3(256), 0, st, a, ja, jb);
      else hipLaunchKernelGGL((piece_kernel<NA, NB, false>), grid, dim3(256), 0, st, a, ja, jb);
    });
  });
  JoinArgs j{};
  j.l = p.l;
  j.offsets = q.rows.offsets;
  j.tiles = q.rows.tiles;
  j.list = p.list;
  j.part = sums;
  j.slot = p.slot;
  j.off[0] = 0;
  j.off[1] = (long)p.R * d.K;
  j.per[0] = q.dA != nullptr ? (long)p.R * d.K : 0;
  j.per[1] = q.dB != nullptr ? (long)d.N * d.r : 0;
  j.out[0] = q.dA;
  j.out[1] = q.dB;
  hipLaunchKernelGGL(join_kernel, dim3((unsigned)((j.per[0] + j.per[1] + 1023) / 1024), d.n), dim3(256), 0, st, j);
  return hipGetLastError();
}

}  // namespace oft
