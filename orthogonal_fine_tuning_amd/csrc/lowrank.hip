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
// backward runs them on transposed copies of the factors.  `pieces` forms the
// sums over rows.  Everything is bound by the bytes of x, y, dy and dx, so the
// products take whatever keeps those moving: 16 x 16 x 32 matrix steps (ranks
// and tiles of single decoded rows are small), operands straight from global
// memory where both run along the contraction.
//
// Precision: bf16 factors and activations are matrix operands as they are.
// fp32 values (v, u, fp32 activations) are split into bf16 parts whose sum is
// the value (split_bf16): all three where the result is fp32, two where it is
// rounded to bf16, whose half step of 2^-9 hides the 2^-16 left out.
#include "adapter_device.h"
#include "gemm_nn.h"
#include "oft_prof.h"

namespace oft {
namespace {

// ------------------------------------------------------------------- down
// part[split][row][j] = sum over the split's columns of src[row] W[j], the
// split sums added by whoever reads them.  A job is up to 64 of a segment's
// output columns, or of all of them where the rows of src are whole.
struct DownArgs {
  RowLists l;
  RowOrder rows;
  const void* src;
  long lds;
  const uint16_t* w;
  long w_a;  // elements of an adapter's matrices
  float* part;
  int R;       // columns of part
  int nsplit;
  int n_seg, r, per;  // r output columns a segment (R when whole), `per` a job
  int jobs_per_seg;
  bool whole;
  int K;
  int seg_at[MAX_SEG + 1];
};

template <int TM, int NG, bool F32>
__global__ __launch_bounds__(256) void down_kernel(DownArgs a) {
  constexpr int P = Oct<F32>::P, XG = TM / 16;
  __shared__ __attribute__((aligned(16))) float red[2][XG * NG * 4][64];
  const int split = blockIdx.y, job = blockIdx.z;
  int4 e;
  if (!list_entry(a.l, a.rows.tiles, TM == 16 ? LIST_16 : LIST_64, blockIdx.x, e) || e.x < 0) return;
  const int seg = job / a.jobs_per_seg, sub = job % a.jobs_per_seg;
  const int col0 = a.whole ? 0 : a.seg_at[seg];
  const int len = a.whole ? a.K : a.seg_at[seg + 1] - col0;
  const int jw = sub * a.per, nj = min(a.per, a.r - jw);  // rows of this segment's matrix
  const uint16_t* w = a.w + (size_t)e.x * a.w_a + (a.whole ? 0 : (size_t)a.r * col0) + (size_t)jw * len;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  // the split's columns in steps of 64, dealt to the four waves in turn
  const int steps = (len + 63) / 64, per = (steps + a.nsplit - 1) / a.nsplit;
  const int s0 = split * per, s1 = min(steps, s0 + per);

  size_t xrow[XG];
  int row[XG];
#pragma unroll
  for (int i = 0; i < XG; ++i) {
    row[i] = row_at(a.l, a.rows.order, e.y + min(16 * i + l16, e.z - 1));
    xrow[i] = (size_t)row[i] * a.lds + col0;
  }
  size_t wrow[NG];
#pragma unroll
  for (int j = 0; j < NG; ++j) wrow[j] = (size_t)min(16 * j + l16, nj - 1) * len;

  f32x4 acc[XG][NG];
#pragma unroll
  for (int i = 0; i < XG; ++i)
#pragma unroll
    for (int j = 0; j < NG; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  Oct<F32> x[XG][2];
  uint4 wv[NG][2];
  // a lane's 16 columns of a step are contiguous: 32 bytes of bf16
  auto load = [&](int s) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int k = 64 * s + 16 * g + 8 * t;
      const bool ok = k < len;  // (segments are multiples of 16)
#pragma unroll
      for (int i = 0; i < XG; ++i) {
        if (ok) x[i][t].load(a.src, xrow[i] + k);
        else x[i][t].zero();
      }
#pragma unroll
      for (int j = 0; j < NG; ++j) wv[j][t] = ok ? *reinterpret_cast<const uint4*>(w + wrow[j] + k) : zero4();
    }
  };
  int s = s0 + wave;
  if (s < s1) load(s);
  for (; s < s1; s += 4) {
    Oct<F32> xc[XG][2];
    uint4 wc[NG][2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int i = 0; i < XG; ++i) xc[i][t] = x[i][t];
#pragma unroll
      for (int j = 0; j < NG; ++j) wc[j][t] = wv[j][t];
    }
    if (s + 4 < s1) load(s + 4);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < XG; ++i) {
        uint4 xp[P];
        xc[i][t].parts(xp);
#pragma unroll
        for (int j = 0; j < NG; ++j)
#pragma unroll
          for (int p = P - 1; p >= 0; --p) acc[i][j] = mfma16(as_bf16x8(wc[j][t]), as_bf16x8(xp[p]), acc[i][j]);
      }
  }
  // the four waves' sums, in a fixed order: (0 + 2) + (1 + 3)
  if (wave >= 2) {
#pragma unroll
    for (int i = 0; i < XG; ++i)
#pragma unroll
      for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) red[wave - 2][(i * NG + j) * 4 + c][lane] = acc[i][j][c];
  }
  __syncthreads();
  if (wave < 2) {
#pragma unroll
    for (int i = 0; i < XG; ++i)
#pragma unroll
      for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][j][c] += red[wave][(i * NG + j) * 4 + c][lane];
  }
  __syncthreads();
  if (wave == 1) {
#pragma unroll
    for (int i = 0; i < XG; ++i)
#pragma unroll
      for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) red[0][(i * NG + j) * 4 + c][lane] = acc[i][j][c];
  }
  __syncthreads();
  if (wave != 0) return;
  // lane: row l16 of each 16, four consecutive output columns
#pragma unroll
  for (int i = 0; i < XG; ++i) {
    if (16 * i + l16 >= e.z) continue;
    float* out = a.part + ((size_t)split * a.l.T + row[i]) * a.R + (a.whole ? 0 : seg * a.r) + jw;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const int c0 = 16 * j + 4 * g;
      if (c0 < nj) {  // (ranks are multiples of 8)
        float4 v;
        v.x = acc[i][j][0] + red[0][(i * NG + j) * 4 + 0][lane];
        v.y = acc[i][j][1] + red[0][(i * NG + j) * 4 + 1][lane];
        v.z = acc[i][j][2] + red[0][(i * NG + j) * 4 + 2][lane];
        v.w = acc[i][j][3] + red[0][(i * NG + j) * 4 + 3][lane];
        *reinterpret_cast<float4*>(out + c0) = v;
      }
    }
  }
}

// --------------------------------------------------------------------- up
// out[row][c] = base[row][c] + scale sum_k v[row][k] W[c][k]: a wave per 64
// columns of one segment and TM rows.  The lane's operand row of W is column
// 16 (l / 4 % 4) + 4 m + l % 4 of the 64 in matrix step m, so that its results
// of the four steps are 16 consecutive columns of one row.
struct UpArgs {
  RowLists l;
  RowOrder rows;
  const float* part;  // [nsplit][T][R], summed here
  int nsplit, R, r;   // r: the contraction, from column seg * r of part
  const uint16_t* w;  // [n][C][r]
  long w_a;
  const float* scale;
  const void* base;
  void* out;
  int C;       // columns
  float* v;    // [T][R], the summed part (NULL: not kept)
  int n_seg, cblocks;
  int seg_at[MAX_SEG + 1], block_at[MAX_SEG + 1];  // columns and 64-column blocks before each segment
};

template <int TM, bool F32>
__global__ __launch_bounds__(256) void up_kernel(UpArgs a) {
  constexpr int P = F32 ? 3 : 2, XG = TM / 16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  const int wgs = (a.cblocks + 3) / 4;
  const int tile = blockIdx.x / wgs, cb = (blockIdx.x % wgs) * 4 + wave;
  int4 e;
  if (cb >= a.cblocks || !list_entry(a.l, a.rows.tiles, TM == 16 ? LIST_16 : LIST_64, tile, e)) return;
  int seg = 0;
#pragma unroll
  for (int i = 1; i < MAX_SEG; ++i) seg += i < a.n_seg && cb >= a.block_at[i];
  int seg_lo = 0, seg_hi = 0, blk_lo = 0;
#pragma unroll
  for (int i = 0; i < MAX_SEG; ++i)
    if (i == seg) {
      seg_lo = a.seg_at[i];
      seg_hi = a.seg_at[i + 1];
      blk_lo = a.block_at[i];
    }
  const int n0 = seg_lo + 64 * (cb - blk_lo);
  const bool col_ok = n0 + 16 * g < seg_hi;  // this lane's 16 columns (segments are multiples of 16)

  Oct<F32> y[XG][2];
  size_t at[XG];
  int row[XG];
#pragma unroll
  for (int i = 0; i < XG; ++i) {
    row[i] = row_at(a.l, a.rows.order, e.y + min(16 * i + l16, e.z - 1));
    at[i] = (size_t)row[i] * a.C + n0 + 16 * g;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (col_ok && a.base != nullptr) y[i][h].load(a.base, at[i] + 8 * h);
      else y[i][h].zero();
    }
  }
  if (e.x < 0) {  // rows of the base model
    if (a.base != a.out && col_ok) {
#pragma unroll
      for (int i = 0; i < XG; ++i)
        if (16 * i + l16 < e.z)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (F32) {
              float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at[i] + 8 * h);
              o[0] = y[i][h].a;
              o[1] = y[i][h].b;
            } else {
              *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at[i] + 8 * h) = y[i][h].u;
            }
          }
    }
    if (a.v != nullptr && n0 == seg_lo) {
      for (int k = 8 * g; k < a.r; k += 32)
#pragma unroll
        for (int i = 0; i < XG; ++i)
          if (16 * i + l16 < e.z) {
            float4* o = reinterpret_cast<float4*>(a.v + (size_t)row[i] * a.R + seg * a.r + k);
            o[0] = o[1] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
    }
    return;
  }
  const uint16_t* w = a.w + (size_t)e.x * a.w_a;
  size_t wrow[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) wrow[m] = (size_t)min(n0 + 16 * (l16 >> 2) + 4 * m + (l16 & 3), seg_hi - 1) * a.r;

  f32x4 acc[XG][4];
#pragma unroll
  for (int i = 0; i < XG; ++i)
#pragma unroll
    for (int m = 0; m < 4; ++m) acc[i][m] = f32x4{0.f, 0.f, 0.f, 0.f};
  const size_t plane = (size_t)a.l.T * a.R;
  for (int k0 = 0; k0 < a.r; k0 += 32) {
    const int k = k0 + 8 * g;
    const bool ok = k < a.r;
    uint4 wv[4];
#pragma unroll
    for (int m = 0; m < 4; ++m) wv[m] = ok ? *reinterpret_cast<const uint4*>(w + wrow[m] + k) : zero4();
#pragma unroll
    for (int i = 0; i < XG; ++i) {
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (ok) {
        const float* p = a.part + (size_t)row[i] * a.R + seg * a.r + k;
        for (int s = 0; s < a.nsplit; ++s, p += plane) {
          const float4 c = reinterpret_cast<const float4*>(p)[0], d = reinterpret_cast<const float4*>(p)[1];
          v[0] += c.x;
          v[1] += c.y;
          v[2] += c.z;
          v[3] += c.w;
          v[4] += d.x;
          v[5] += d.y;
          v[6] += d.z;
          v[7] += d.w;
        }
        if (a.v != nullptr && n0 == seg_lo && 16 * i + l16 < e.z) {
          float4* o = reinterpret_cast<float4*>(a.v + (size_t)row[i] * a.R + seg * a.r + k);
          o[0] = make_float4(v[0], v[1], v[2], v[3]);
          o[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
      uint4 vp[P];
      split_bf16x8<P>(v, vp);
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int p = P - 1; p >= 0; --p) acc[i][m] = mfma16(as_bf16x8(wv[m]), as_bf16x8(vp[p]), acc[i][m]);
    }
  }
  const float sc = a.scale[e.x];
#pragma unroll
  for (int i = 0; i < XG; ++i) {
    if (!col_ok || 16 * i + l16 >= e.z) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float o[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) o[c] = sc * acc[i][2 * h + c / 4][c % 4];
      if constexpr (F32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at[i] + 8 * h);
        q[0] = make_float4(y[i][h].a.x + o[0], y[i][h].a.y + o[1], y[i][h].a.z + o[2], y[i][h].a.w + o[3]);
        q[1] = make_float4(y[i][h].b.x + o[4], y[i][h].b.y + o[5], y[i][h].b.z + o[6], y[i][h].b.w + o[7]);
      } else {
        const uint32_t b[4] = {y[i][h].u.x, y[i][h].u.y, y[i][h].u.z, y[i][h].u.w};
        uint32_t q[4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          q[c] = pack_bf16x2(bf16_to_f32(b[c] & 0xFFFF) + o[2 * c], bf16_to_f32(b[c] >> 16) + o[2 * c + 1]);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at[i] + 8 * h) = make_uint4(q[0], q[1], q[2], q[3]);
      }
    }
  }
}

// -------------------------------------------------------------- transposes
// The factors of the adapters in use, transposed: matrix s of an adapter is
// [rows_s, cols] at element off_s and becomes [cols, rows_s] at the same
// place.  64 x 64 tiles through LDS.
struct TransposeArgs {
  const int* offsets;
  const uint16_t* in;
  uint16_t* out;
  long per;  // elements of an adapter
  int n_seg, cols;
  int at[MAX_SEG + 1], tile_at[MAX_SEG + 1];  // rows, 64-row tiles before each matrix
};

__device__ __forceinline__ void transpose_tile(const TransposeArgs& a, int tile, int ad, uint16_t (&t)[64][66]) {
  const int ct = (a.cols + 63) / 64;
  const int rt = tile / ct, c0 = (tile % ct) * 64;
  int lo = 0, hi = 0, r0 = 0;
#pragma unroll
  for (int i = 0; i < MAX_SEG; ++i)
    if (i < a.n_seg && rt >= a.tile_at[i]) {
      lo = a.at[i];
      hi = a.at[i + 1];
      r0 = 64 * (rt - a.tile_at[i]);
    }
  const uint16_t* in = a.in + (size_t)ad * a.per + (size_t)lo * a.cols;
  uint16_t* out = a.out + (size_t)ad * a.per + (size_t)lo * a.cols;
  const int rows = hi - lo;
  for (int i = threadIdx.x; i < 64 * 8; i += 256) {
    const int r = r0 + i / 8, c = c0 + 8 * (i % 8);
    if (r < rows && c < a.cols) {
      const uint4 u = *reinterpret_cast<const uint4*>(in + (size_t)r * a.cols + c);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 8; ++j) t[8 * (i % 8) + j][i / 8] = (uint16_t)(w[j / 2] >> (16 * (j % 2)));
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 8; i += 256) {
    const int c = c0 + i / 8, r = r0 + 8 * (i % 8);
    if (c < a.cols && r < rows) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = t[i / 8][8 * (i % 8) + 2 * j] | ((uint32_t)t[i / 8][8 * (i % 8) + 2 * j + 1] << 16);
      *reinterpret_cast<uint4*>(out + (size_t)c * rows + r) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

__global__ __launch_bounds__(256) void transpose_kernel(TransposeArgs a, int tiles_a, TransposeArgs b, int tiles_b) {
  __shared__ uint16_t t[64][66];
  const int ad = blockIdx.y;
  if (a.offsets[ad] >= a.offsets[ad + 1]) return;
  if ((int)blockIdx.x < tiles_a) transpose_tile(a, blockIdx.x, ad, t);
  else if ((int)blockIdx.x < tiles_a + tiles_b) transpose_tile(b, blockIdx.x - tiles_a, ad, t);
}

// ------------------------------------------------------------------ pieces
// Sums over an adapter's rows: out[j][c] = scale sum_rows U[row][j] X[row][c]
// for 256 columns of X and up to 64 of U, over one piece of the adapter's
// rows.  Both operands run along the rows here: tiles of 32 rows go to LDS in
// row order and are read with the transposing LDS load.  U is fp32 in three
// parts; so is X where it is fp32 (products of parts whose scales differ by
// 2^-24 or more are left out).
constexpr int PC = 256, PR = 32;  // columns, rows of a step
constexpr int LDX = PC + 16;      // LDS row: 16 elements more, so that four rows of a transposing read fall in four banks' groups

struct PieceJob {
  const void* x;
  long ldx;
  const float* u;  // summed over nsplit planes
  int nsplit;
  float* out;      // [n][...], element (j, c) at j so_j + c so_c
  long out_a;
  long part_off;   // this sum's place in a partial slot
  int so_j, so_c;
  int blocks;      // column blocks of one segment's columns, over all segments
  int nj, njc;     // columns of U a segment, and chunks of 64 of them
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

template <int NJ, bool F32>
__device__ __forceinline__ void piece(const PieceArgs& a, const PieceJob& q, int4 e, int job, uint16_t* xs, uint16_t* us) {
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

  f32x4 acc[NJ][4];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[j][c] = f32x4{0.f, 0.f, 0.f, 0.f};

  // thread: 8 columns of rows tid / 32 + 8 i of a step; U: 4 columns of row
  // tid / (4 NJ) (+ 64 / NJ ...)
  const int xc = c0 + 8 * (tid & 31), xr = tid >> 5;
  const bool xok = xc < c_hi;
  constexpr int UT = 4 * NJ, UR = 256 / UT, UI = (PR + UR - 1) / UR;
  const int uc = 4 * (tid % UT), ur = tid / UT;
  const size_t plane = (size_t)a.l.T * a.R;
  Oct<F32> x[4];
  float4 u[UI];
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + xr + 8 * i;
      if (r < e.z && xok) x[i].load(q.x, (size_t)row_at(a.l, a.rows.order, e.y + r) * q.ldx + xc);
      else x[i].zero();
    }
#pragma unroll
    for (int i = 0; i < UI; ++i) {
      u[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      const int r = r0 + ur + UR * i;
      if (ur + UR * i < PR && r < e.z && uc < nj) {
        const float* p = q.u + (size_t)row_at(a.l, a.rows.order, e.y + r) * a.R + ju + uc;
        for (int s = 0; s < q.nsplit; ++s, p += plane) {
          const float4 v = *reinterpret_cast<const float4*>(p);
          u[i].x += v.x;
          u[i].y += v.y;
          u[i].z += v.z;
          u[i].w += v.w;
        }
      }
    }
  };
  load(0);
  for (int r0 = 0; r0 < e.z; r0 += PR) {
    __syncthreads();  // the last step's reads are done
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 p[PX];
      x[i].parts(p);
#pragma unroll
      for (int k = 0; k < PX; ++k)
        *reinterpret_cast<uint4*>(xs + (k * PR + xr + 8 * i) * LDX + 8 * (tid & 31)) = p[k];
    }
#pragma unroll
    for (int i = 0; i < UI; ++i)
      if (ur + UR * i < PR) {
        const float v[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
        uint32_t h[4][3];
#pragma unroll
        for (int k = 0; k < 4; ++k) split_bf16<3>(v[k], h[k]);
#pragma unroll
        for (int p = 0; p < 3; ++p)
          *reinterpret_cast<uint2*>(us + (p * PR + ur + UR * i) * LDU + uc) =
              make_uint2(h[0][p] | (h[1][p] << 16), h[2][p] | (h[3][p] << 16));
      }
    __syncthreads();
    if (r0 + PR < e.z) load(r0 + PR);
    // lane l16 of group g: rows 8 g .. 8 g + 7 of column l16 of 16
    const int tr = 8 * g + (l16 >> 2), tc = 4 * (l16 & 3);
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
            if (p + k <= 2) acc[j][c] = mfma16(uv, xv[c][k], acc[j][c]);
      }
  }
  // lane: column l16 of 16, rows (of U^T) 4 g .. 4 g + 3 of 16
  const float sc = a.scale[e.x];
  float* out = e.w < 0 ? q.out + (size_t)e.x * q.out_a : a.part + (size_t)e.w * a.slot + q.part_off;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int jj = 16 * j + 4 * g;
    if (jj >= nj) continue;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int col = c0 + 64 * wave + 16 * c + l16;
      if (col >= c_hi) continue;
      float* o = out + (size_t)(j0 + jj) * q.so_j + (size_t)col * q.so_c;
      if (q.so_j == 1) {
        *reinterpret_cast<float4*>(o) = make_float4(sc * acc[j][c][0], sc * acc[j][c][1], sc * acc[j][c][2], sc * acc[j][c][3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) o[(size_t)k * q.so_j] = sc * acc[j][c][k];
      }
    }
  }
}

template <int NA, int NB, bool F32>
__global__ __launch_bounds__(256) void piece_kernel(PieceArgs a, PieceJob qa, PieceJob qb) {
  constexpr int NJ = NA > NB ? NA : NB;
  __shared__ __attribute__((aligned(16))) uint16_t xs[Oct<F32>::P * PR * LDX];
  __shared__ __attribute__((aligned(16))) uint16_t us[3 * PR * (NJ * 16 + 16)];
  int4 e;
  if (!list_entry(a.l, a.rows.tiles, a.list, blockIdx.y, e) || e.x < 0) return;
  e.w = min(e.w, RowLists::slots(a.list) - 1);
  const int ja = qa.blocks * qa.njc;
  if ((int)blockIdx.x < ja) piece<NA, F32>(a, qa, e, blockIdx.x, xs, us);
  else piece<NB, false>(a, qb, e, blockIdx.x - ja, xs, us);
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
  const int first = a.tiles[a.l.part_at(a.list) + ad];
  const int slots = min(pieces, RowLists::slots(a.list) - first);
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
// has few), else 64.
int tile_rows(int T) { return T <= 1024 ? 16 : 64; }

struct DownPlan {
  int per, jobs_per_seg, jobs, nsplit, ng;
};
// len: the longest contraction; r columns for each of n_seg segments
DownPlan plan_down(const RowLists& l, int tm, int len, int r, int n_seg) {
  DownPlan p;
  const int groups = (r + 15) / 16;
  p.jobs_per_seg = (groups + 3) / 4;
  p.ng = (groups + p.jobs_per_seg - 1) / p.jobs_per_seg;
  p.per = 16 * p.ng;
  p.jobs = n_seg * p.jobs_per_seg;
  // enough workgroups for two a CU where the tiles alone do not give them,
  // each with a step of 64 columns for every wave
  const long tiles = (l.T + tm - 1) / tm;
  long want = (512 + tiles * p.jobs - 1) / (tiles * p.jobs);
  const long most = len / 256 > 1 ? len / 256 : 1;
  want = want < 1 ? 1 : want > most ? most : want;
  p.nsplit = (int)want;
  return p;
}

struct Plan {
  RowLists l;
  int tm, R;
  DownPlan down;
  int list;
  size_t part, at, bt, sums, bytes;
  long slot;
};
Plan plan_of(const LowrankDims& d, bool bwd) {
  Plan p;
  p.l = RowLists{d.T, d.n};
  p.tm = tile_rows(d.T);
  p.R = d.n_seg * d.r;
  int longest = 0;
  for (int i = 0; i < d.n_seg; ++i) longest = d.seg[i] > longest ? d.seg[i] : longest;
  p.down = bwd ? plan_down(p.l, p.tm, longest, d.r, d.n_seg) : plan_down(p.l, p.tm, d.K, p.R, 1);
  p.part = 0;
  p.bytes = up256(4 * (size_t)p.down.nsplit * d.T * p.R);
  p.at = p.bt = p.sums = 0;
  p.slot = (long)p.R * d.K + (long)d.N * d.r;
  p.list = LIST_SHORT;
  if (bwd) {
    p.at = p.bytes;
    p.bt = p.at + up256(2 * (size_t)d.n * p.R * d.K);
    p.sums = p.bt + up256(2 * (size_t)d.n * d.N * d.r);
    // column blocks: pieces of a quarter of the rows where they alone nearly
    // fill the chip
    const long blocks = (d.K + PC - 1) / PC + (d.N + PC - 1) / PC;
    p.list = blocks >= 128 ? LIST_LONG : LIST_SHORT;
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

void run_down(const Plan& p, const DownArgs& a, bool f32, hipStream_t st) {
  const dim3 grid(p.l.cap(p.tm == 16 ? LIST_16 : LIST_64), p.down.nsplit, p.down.jobs);
  groups_of(p.down.ng, [&](auto ng) {
    constexpr int NG = decltype(ng)::value;
    if (p.tm == 16) {
      if (f32) hipLaunchKernelGGL((down_kernel<16, NG, true>), grid, dim3(256), 0, st, a);
      else hipLaunchKernelGGL((down_kernel<16, NG, false>), grid, dim3(256), 0, st, a);
    } else {
      if (f32) hipLaunchKernelGGL((down_kernel<64, NG, true>), grid, dim3(256), 0, st, a);
      else hipLaunchKernelGGL((down_kernel<64, NG, false>), grid, dim3(256), 0, st, a);
    }
  });
}

void run_up(const Plan& p, UpArgs a, bool f32, hipStream_t st) {
  a.block_at[0] = 0;
  for (int i = 0; i < MAX_SEG; ++i)
    a.block_at[i + 1] = i < a.n_seg ? a.block_at[i] + (a.seg_at[i + 1] - a.seg_at[i] + 63) / 64 : a.block_at[i];
  a.cblocks = a.block_at[a.n_seg];
  const dim3 grid((unsigned)p.l.cap(p.tm == 16 ? LIST_16 : LIST_64) * ((a.cblocks + 3) / 4));
  if (p.tm == 16) {
    if (f32) hipLaunchKernelGGL((up_kernel<16, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((up_kernel<16, false>), grid, dim3(256), 0, st, a);
  } else {
    if (f32) hipLaunchKernelGGL((up_kernel<64, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((up_kernel<64, false>), grid, dim3(256), 0, st, a);
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

int tiles_of(TransposeArgs& t) {
  t.tile_at[0] = 0;
  for (int i = 0; i < MAX_SEG; ++i)
    t.tile_at[i + 1] = i < t.n_seg ? t.tile_at[i] + (t.at[i + 1] - t.at[i] + 63) / 64 : t.tile_at[i];
  return t.tile_at[t.n_seg] * ((t.cols + 63) / 64);
}

}  // namespace

size_t lowrank_ws_bytes(const LowrankDims& d, bool bwd) { return plan_of(d, bwd).bytes; }

hipError_t launch_lowrank_fwd(const LowrankDims& d, const LowrankPtrs& q, char* ws, hipStream_t st) {
  ProfScope prof(st, "lowrank.fwd");
  const Plan p = plan_of(d, false);
  float* part = reinterpret_cast<float*>(ws + p.part);
  DownArgs a{};
  a.l = p.l;
  a.rows = q.rows;
  a.src = q.x;
  a.lds = d.K;
  a.w = q.A;
  a.w_a = (long)p.R * d.K;
  a.part = part;
  a.R = p.R;
  a.nsplit = p.down.nsplit;
  a.n_seg = 1;
  a.r = p.R;
  a.per = p.down.per;
  a.jobs_per_seg = p.down.jobs_per_seg;
  a.whole = true;
  a.K = d.K;
  run_down(p, a, d.f32, st);
  UpArgs b{};
  b.l = p.l;
  b.rows = q.rows;
  b.part = part;
  b.nsplit = p.down.nsplit;
  b.R = p.R;
  b.r = d.r;
  b.w = q.B;
  b.w_a = (long)d.N * d.r;
  b.scale = q.scale;
  b.base = q.y_base;
  b.out = q.y;
  b.C = d.N;
  b.v = q.v;
  b.n_seg = d.n_seg;
  segments(d, b.seg_at);
  run_up(p, b, d.f32, st);
  return hipGetLastError();
}

hipError_t launch_lowrank_bwd(const LowrankDims& d, const LowrankGradPtrs& q, char* ws, hipStream_t st) {
  ProfScope prof(st, "lowrank.bwd");
  const Plan p = plan_of(d, true);
  float* part = reinterpret_cast<float*>(ws + p.part);
  uint16_t* at = reinterpret_cast<uint16_t*>(ws + p.at);
  uint16_t* bt = reinterpret_cast<uint16_t*>(ws + p.bt);
  float* sums = reinterpret_cast<float*>(ws + p.sums);

  // (without rows only the gradients' zeros are left to write)
  if (d.T > 0 && (q.dx != nullptr || q.dA != nullptr)) {
    TransposeArgs ta{}, tb{};
    ta.offsets = tb.offsets = q.rows.offsets;
    ta.in = q.A;
    ta.out = at;
    ta.per = (long)p.R * d.K;
    ta.n_seg = 1;
    ta.cols = d.K;
    one_segment(p.R, ta.at);
    tb.in = q.B;
    tb.out = bt;
    tb.per = (long)d.N * d.r;
    tb.n_seg = d.n_seg;
    tb.cols = d.r;
    segments(d, tb.at);
    const int na = q.dx != nullptr ? tiles_of(ta) : 0, nb = tiles_of(tb);
    hipLaunchKernelGGL(transpose_kernel, dim3(na + nb, d.n), dim3(256), 0, st, ta, na, tb, nb);
    DownArgs a{};
    a.l = p.l;
    a.rows = q.rows;
    a.src = q.dy;
    a.lds = d.N;
    a.w = bt;
    a.w_a = (long)d.N * d.r;
    a.part = part;
    a.R = p.R;
    a.nsplit = p.down.nsplit;
    a.n_seg = d.n_seg;
    a.r = d.r;
    a.per = p.down.per;
    a.jobs_per_seg = p.down.jobs_per_seg;
    a.whole = false;
    segments(d, a.seg_at);
    run_down(p, a, false, st);
  }
  if (d.T > 0 && q.dx != nullptr) {
    UpArgs b{};
    b.l = p.l;
    b.rows = q.rows;
    b.part = part;
    b.nsplit = p.down.nsplit;
    b.R = b.r = p.R;
    b.w = at;
    b.w_a = (long)p.R * d.K;
    b.scale = q.scale;
    b.base = q.dx_base;
    b.out = q.dx;
    b.C = d.K;
    b.n_seg = 1;
    one_segment(d.K, b.seg_at);
    run_up(p, b, d.f32, st);
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
  ja.u = part;
  ja.nsplit = p.down.nsplit;
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
  jb.nsplit = 1;
  jb.out = q.dB;
  jb.out_a = (long)d.N * d.r;
  jb.part_off = (long)p.R * d.K;
  jb.so_j = 1;
  jb.so_c = d.r;
  jb.n_seg = d.n_seg;
  jb.nj = d.r;
  segments(d, jb.seg_at);
  blocks_of(jb, PC);
  // columns of U a workgroup takes: up to 64, evenly
  const int ga = (p.R + 15) / 16, gb = (d.r + 15) / 16;
  ja.njc = (ga + 3) / 4;
  jb.njc = (gb + 3) / 4;
  const int na = (ga + ja.njc - 1) / ja.njc, nb = (gb + jb.njc - 1) / jb.njc;
  if (q.dA == nullptr) ja.blocks = 0;
  if (q.dB == nullptr) jb.blocks = 0;
  const dim3 grid(ja.blocks * ja.njc + jb.blocks * jb.njc, p.l.cap(p.list));
  if (d.T > 0) groups_of(na, [&](auto va) {
    groups_of(nb, [&](auto vb) {
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
