// Block rotations of many requests' orthogonal adapters after a shared
// projection, and their gradients (oft_rotate_fwd / oft_rotate_bwd in oft.h).
//
//   forward   y_blk = R_j z_blk                        (the row's own R)
//   backward  dz_blk = R_j^T dy_blk,
//             S_j = sum_rows dy_blk y_blk^T,
//             Gq = (R_j^T + I) S_j (I + R_j) / 2,  dp_il = Gq_il - Gq_li
// (as in the linear layer's backward).  2 b operations per element of a row:
// bound by the bytes of the rows, and for single decoded rows by those of the
// rotations.  A wave takes 32 channels of a tile of rows and keeps their
// rotation in registers as a matrix operand (two 16-channel blocks as one
// block-diagonal operand); the channels of a lane's operand are also those of
// its result, eight consecutive ones of a row.
//
// fp32 rows are split into three bf16 parts whose sum is the value; bf16 rows
// and rotations are operands as they are.
#include "adapter_device.h"
#include "gemm_nn.h"
#include "oft_prof.h"

namespace oft {
namespace {

// Rotation operands of channels n0 .. n0 + 31 (pack `which`: 0 R, 1 R^T), for
// 16 rows at a time: operand row i of matrix step m is channel
// 8 (i / 4) + 4 m + i % 4, contraction item p of lane group g channel 8 g + p, so
// that a lane's results of the two steps are the eight channels that it
// brought itself.
template <int B>
__device__ __forceinline__ void load_rotation(const uint16_t* __restrict__ rops, int n0, int which, int l16, int g,
                                              uint4 (&o)[2]) {
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int c = 8 * (l16 >> 2) + 4 * m + (l16 & 3);
    if constexpr (B == 32)
      o[m] = *reinterpret_cast<const uint4*>(rops + (size_t)(n0 / 32) * 2048 + which * 1024 + c * 32 + 8 * g);
    else
      o[m] = (c >> 4) == (g >> 1) ? *reinterpret_cast<const uint4*>(rops + (size_t)(n0 / 16 + (g >> 1)) * 512 +
                                                                    which * 256 + (c & 15) * 16 + 8 * (g & 1))
                                  : zero4();
  }
}

// Of two 16-channel blocks, lane groups 0 and 1 bring the first and take its
// results, 2 and 3 the second.  Each block is a product of its own, with zeros
// in place of the other's rows: a NaN or an infinity times the zeros beside a
// block's rotation would be NaN.  (us with both blocks in one product and with
// two: 64 rows of 6144 channels 4.6 and 4.7, 8192 rows of 19456 channels 120
// and 119, sums of 4096 such rows 96 and 97, of 1501 fp32 rows of 6144 22.6 and
// 24.1)
template <int B, bool F32>
__device__ __forceinline__ void rotate(const uint4 (&rot)[2], const Oct<F32>& z, int g, f32x4 (&o)[2]) {
  constexpr int P = Oct<F32>::P;
  uint4 p[P];
  z.parts(p);
  const bool second = g >= 2;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    o[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    if constexpr (B == 32) {
#pragma unroll
      for (int k = P - 1; k >= 0; --k) o[m] = mfma16(as_bf16x8(rot[m]), as_bf16x8(p[k]), o[m]);
    } else {
      f32x4 q = o[m];
#pragma unroll
      for (int k = P - 1; k >= 0; --k) {
        o[m] = mfma16(as_bf16x8(rot[m]), as_bf16x8(second ? zero4() : p[k]), o[m]);
        q = mfma16(as_bf16x8(rot[m]), as_bf16x8(second ? p[k] : zero4()), q);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) o[m][i] = second ? q[i] : o[m][i];
    }
  }
}

__device__ __forceinline__ uint4 pack8(const f32x4 (&o)[2]) {
  return make_uint4(pack_bf16x2(o[0][0], o[0][1]), pack_bf16x2(o[0][2], o[0][3]), pack_bf16x2(o[1][0], o[1][1]),
                    pack_bf16x2(o[1][2], o[1][3]));
}

// ------------------------------------------------------------------ rows
// A wave per TM rows and 32 channels: decoded rows, and rows of fp32.
template <int TM, int B, bool F32>
__global__ __launch_bounds__(256) void rotate_kernel(RowLists l, RowOrder rows, const void* z,
                                                     const uint16_t* __restrict__ rops, int N, int which, void* y) {
  constexpr int XG = TM / 16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  const int wgs = (N + 127) / 128;
  const int n0 = (blockIdx.x % wgs) * 128 + 32 * wave;
  int4 e;
  if (n0 >= N || !list_entry(l, rows.tiles, TM == 16 ? LIST_16 : LIST_64, blockIdx.x / wgs, e)) return;
  uint4 rot[2];  // (does not wait for the rows' numbers)
  if (e.x >= 0) load_rotation<B>(rops + (size_t)e.x * N * B * 2, n0, which, l16, g, rot);
  Oct<F32> x[XG];
  size_t at[XG];
#pragma unroll
  for (int i = 0; i < XG; ++i) {
    at[i] = (size_t)row_at(l, rows.order, e.y + min(16 * i + l16, e.z - 1)) * N + n0 + 8 * g;
    x[i].load(z, at[i]);
  }
  if (e.x >= 0) {
#pragma unroll
    for (int i = 0; i < XG; ++i) {
      f32x4 o[2];
      rotate<B, F32>(rot, x[i], g, o);
      if constexpr (F32) {
        x[i].a = make_float4(o[0][0], o[0][1], o[0][2], o[0][3]);
        x[i].b = make_float4(o[1][0], o[1][1], o[1][2], o[1][3]);
      } else {
        x[i].u = pack8(o);
      }
    }
  } else if (y == z) {
    return;
  }
#pragma unroll
  for (int i = 0; i < XG; ++i)
    if (16 * i + l16 < e.z) x[i].store(y, at[i]);
}

// bf16 rows in tiles of 64: a wave per tile and 64 channels, through its own
// LDS tile.
constexpr int RW = 2;  // waves of a workgroup; they share nothing

template <int B, bool STREAM>
__global__ __launch_bounds__(64 * RW) void rotate_tile_kernel(RowLists l, RowOrder rows, const uint16_t* z,
                                                          const uint16_t* __restrict__ rops, int N, int which,
                                                          uint16_t* y) {
  __shared__ __attribute__((aligned(16))) char lds[RW][WaveTile::BYTES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  const int wgs = (N + 64 * RW - 1) / (64 * RW);
  const int n0 = ((blockIdx.x % wgs) * RW + wave) * 64;
  int4 e;
  if (n0 >= N || !list_entry(l, rows.tiles, LIST_64, blockIdx.x / wgs, e)) return;
  const int c = n0 + 8 * (lane & 7);  // (N is a multiple of 32: a piece is inside or not)
  int row[8];
  tile_rows8(l, rows.order, e, lane, row);
  Oct<false> x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c < N) x[i].load<STREAM>(z, (size_t)row[i] * N + c);
    else x[i].zero();
  if (e.x >= 0) {
    uint4 rot[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (n0 + 32 * k < N) load_rotation<B>(rops + (size_t)e.x * N * B * 2, n0 + 32 * k, which, l16, g, rot[k]);
      else rot[k][0] = rot[k][1] = zero4();
    const WaveTile t{lds[wave]};
#pragma unroll
    for (int i = 0; i < 8; ++i) t.by_row(i, lane) = x[i].u;
    wave_order();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        Oct<false> v;
        v.u = t.by_operand(i, 4 * k + g, lane);
        f32x4 o[2];
        rotate<B, false>(rot[k], v, g, o);
        t.by_operand(i, 4 * k + g, lane) = pack8(o);  // (the lane's own 16 bytes)
      }
    wave_order();
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i].u = t.by_row(i, lane);
  } else if (y == z) {
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (8 * i + (lane >> 3) < e.z && c < N) x[i].store<STREAM>(y, (size_t)row[i] * N + c);
}

// ------------------------------------------------------- sums over the rows
// One piece of an adapter's rows and SC channels: dz of every row (dz may be
// NULL, or dy itself), S of the channels' blocks.  Tiles of 32 rows go to LDS in row order;
// S's operands, which run along the rows, are read with the transposing load.
// Rows are fetched two steps ahead.
constexpr int SC = 128, SR = 32, LDS_ROW = SC + 16;

template <int B, bool F32, bool STREAM>
__global__ __launch_bounds__(256, B == 32 && !F32 ? 4 : 1) void rotate_sums_kernel(RowLists l, RowOrder rows, int list,
                                                          const uint16_t* dy, const void* __restrict__ y,
                                                          const float* __restrict__ Rf,
                                                          const uint16_t* __restrict__ rops, int N, uint16_t* dz,
                                                          float* __restrict__ dq, float* __restrict__ part) {
  constexpr int P = Oct<F32>::P, G = 1024 / (B * B), NP = B * (B - 1) / 2;
  constexpr int TILE = SR * LDS_ROW, SROW = 36, SF = SC * SROW;
  constexpr int GRAD = 3 * G * B * (B + 4);  // floats of the Cayley gradient
  constexpr int STEP = (2 + P) * TILE / 2;   // dy, y and dz of a step
  constexpr int FLOATS = STEP > SF + GRAD ? STEP : SF + GRAD;
  constexpr int CL = SC / 8, RL = 256 / CL, NL = SR / RL;  // threads along a row, rows at a time, loads of a thread
  constexpr int CW = SC / 128;                             // groups of 32 channels a wave
  __shared__ __attribute__((aligned(16))) float lds[FLOATS];
  __shared__ int idx[IDX];
  uint16_t* ds = reinterpret_cast<uint16_t*>(lds);
  uint16_t* zs = ds + TILE;
  uint16_t* ys = zs + TILE;

  int4 e;
  if (!list_entry(l, rows.tiles, list, blockIdx.y, e)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l32 = lane & 31, l16 = lane & 15, g = lane >> 5;
  const int n0 = blockIdx.x * SC;
  const int c = n0 + 8 * (tid % CL), r = tid / CL;
  const bool c_ok = c < N;

  if (e.x < 0) {  // rows of the base model: dz = dy, no sums
    if (dz == nullptr || !c_ok || dz == dy) return;
    for (int i = r; i < e.z; i += RL) {
      const size_t at = (size_t)row_at(l, rows.order, e.y + i) * N + c;
      *reinterpret_cast<uint4*>(dz + at) = *reinterpret_cast<const uint4*>(dy + at);
    }
    return;
  }
  uint4 rot[CW][2];
  f32x16 acc[CW], sum[CW];  // of the rows whose numbers are in LDS, and of all
#pragma unroll
  for (int w = 0; w < CW; ++w) {
    rot[w][0] = rot[w][1] = zero4();
    const int nw = n0 + 32 * (wave * CW + w);
    if (dz != nullptr && nw < N) load_rotation<B>(rops + (size_t)e.x * N * B * 2, nw, 1, l16, lane >> 4, rot[w]);
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[w][i] = sum[w][i] = 0.0f;
  }
  // a step's tiles on their way
  struct Tile {
    Oct<false> d[NL];
    Oct<F32> v[NL];
    int row[NL];
  } even, odd;
  int zrow[NL];  // the rows whose dz is in LDS
#pragma unroll
  for (int i = 0; i < NL; ++i) zrow[i] = -1;
  const int at = r * LDS_ROW + 8 * (tid % CL);
  // rows r0 .. of the `rows` whose numbers are in LDS
  auto load = [&](int r0, int rows, Tile& t) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      t.row[i] = -1;
      if (r0 + r + RL * i < rows && c_ok) {
        t.row[i] = idx[r0 + r + RL * i];
        const size_t from = (size_t)t.row[i] * N + c;
        t.d[i].template load<STREAM>(dy, from);
        t.v[i].template load<STREAM>(y, from);
      } else {
        t.d[i].zero();
        t.v[i].zero();
      }
    }
  };
  auto put = [&]() {
    if (dz != nullptr)
#pragma unroll
      for (int i = 0; i < NL; ++i)
        if (zrow[i] >= 0)
          store16<STREAM>(dz + (size_t)zrow[i] * N + c, *reinterpret_cast<const uint4*>(zs + at + RL * i * LDS_ROW));
  };
  auto step = [&](int r0, int rows, Tile& t) {
    __syncthreads();  // the last step's reads are done, its dz complete
    put();
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      zrow[i] = t.row[i];
      *reinterpret_cast<uint4*>(ds + at + RL * i * LDS_ROW) = t.d[i].u;
      uint4 p[P];
      t.v[i].parts(p);
#pragma unroll
      for (int k = 0; k < P; ++k) *reinterpret_cast<uint4*>(ys + k * TILE + at + RL * i * LDS_ROW) = p[k];
    }
    if (r0 + 2 * SR < rows) load(r0 + 2 * SR, rows, t);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < CW; ++w) {
      const int ch = 32 * (wave * CW + w);
      if (dz != nullptr) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int z = (16 * i + l16) * LDS_ROW + ch + 8 * (lane >> 4);
          Oct<false> x;
          x.u = *reinterpret_cast<const uint4*>(ds + z);
          f32x4 o[2];
          rotate<B, false>(rot[w], x, lane >> 4, o);
          *reinterpret_cast<uint4*>(zs + z) = pack8(o);
        }
      }
      // lane l16 of a 16-lane group: 8 rows of one of its 16 channels
#pragma unroll
      for (int k0 = 0; k0 < SR; k0 += 16) {
        const int q0 = (k0 + 8 * g + (l16 >> 2)) * LDS_ROW + ch + 16 * ((lane >> 4) & 1) + 4 * (l16 & 3);
        const uint2 dl = nn::ds_read_tr16(ds + q0), dh = nn::ds_read_tr16(ds + q0 + 4 * LDS_ROW);
        const bf16x8 a = as_bf16x8(make_uint4(dl.x, dl.y, dh.x, dh.y));
#pragma unroll
        for (int k = P - 1; k >= 0; --k) {
          const uint16_t* q = ys + k * TILE + q0;
          const uint2 lo = nn::ds_read_tr16(q), hi = nn::ds_read_tr16(q + 4 * LDS_ROW);
          acc[w] = mfma32(a, as_bf16x8(make_uint4(lo.x, lo.y, hi.x, hi.y)), acc[w]);
        }
      }
    }
  };
  for (int from = 0; from < e.z; from += IDX) {
    const int count = min(IDX, e.z - from);
    __syncthreads();
    fetch_rows(l, rows.order, e.y + from, count, idx);
    __syncthreads();
    load(0, count, even);
    load(SR, count, odd);
    for (int r0 = 0; r0 < count; r0 += 2 * SR) {
      step(r0, count, even);
      if (r0 + SR < count) step(r0 + SR, count, odd);
    }
#pragma unroll
    for (int w = 0; w < CW; ++w)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        sum[w][i] += acc[w][i];
        acc[w][i] = 0.0f;
      }
  }
  __syncthreads();
  put();
  // lane: column l32 of S, rows 8 (i / 4) + 4 g + i % 4
  if (e.w >= 0) {
#pragma unroll
    for (int w = 0; w < CW; ++w) {
      const int nw = n0 + 32 * (wave * CW + w);
      if (nw >= N) break;
      float* out = part + ((size_t)min(e.w, RowLists::slots(list) - 1) * (N / 32) + nw / 32) * 1024;
#pragma unroll
      for (int i = 0; i < 16; ++i) out[(8 * (i / 4) + 4 * g + i % 4) * 32 + l32] = sum[w][i];
    }
    return;
  }
  __syncthreads();
  float* S = lds;  // [SC][SROW]
#pragma unroll
  for (int w = 0; w < CW; ++w)
#pragma unroll
    for (int i = 0; i < 16; ++i) S[(32 * (wave * CW + w) + 8 * (i / 4) + 4 * g + i % 4) * SROW + l32] = sum[w][i];
  const float* R = Rf + (size_t)e.x * N * B;
  float* out = dq + (size_t)e.x * (N / B) * NP;
  for (int h = 0; h < SC / (G * B); ++h) {  // G blocks at a time
    const int b0 = n0 / B + h * G, nb = min(G, N / B - b0);
    if (nb <= 0) break;
    __syncthreads();
    cayley_grad_group<B>(lds + SF, R + (size_t)b0 * B * B, out + (size_t)b0 * NP, nb, tid, [&](int gb, int rr, int cc) {
      const int ch = (h * G + gb) * B;  // channel within the SC
      return *reinterpret_cast<const float4*>(S + (ch + rr) * SROW + (ch & 31) + cc);
    });
  }
}

// dq of the adapters of two or more pieces (their S summed in order), zeros
// for those without rows.
template <int B>
__global__ __launch_bounds__(256) void rotate_join_kernel(RowLists l, RowOrder rows, int list,
                                                          const float* __restrict__ part, const float* __restrict__ Rf,
                                                          int N, float* __restrict__ dq) {
  constexpr int G = 1024 / (B * B), NP = B * (B - 1) / 2;
  __shared__ __attribute__((aligned(16))) float lds[3 * G * B * (B + 4)];
  const int ad = blockIdx.y, tid = threadIdx.x;
  const int pieces = l.count(list, rows.offsets[ad + 1] - rows.offsets[ad]);
  if (pieces == 1) return;
  const int b0 = blockIdx.x * G, nb = min(G, N / B - b0);
  float* out = dq + ((size_t)ad * (N / B) + b0) * NP;
  if (pieces == 0) {
    for (int i = tid; i < nb * NP; i += 256) out[i] = 0.0f;
    return;
  }
  int first;
  const int slots = slots_of(l, rows.tiles, list, ad, pieces, first);
  const size_t plane = (size_t)N * 32;
  cayley_grad_group<B>(lds, Rf + ((size_t)ad * (N / B) + b0) * B * B, out, nb, tid, [&](int gb, int rr, int cc) {
    const int ch = (b0 + gb) * B, in = ch & 31;
    const float* p = part + (size_t)first * plane + (size_t)(ch / 32) * 1024 + (in + rr) * 32 + in + cc;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < slots; ++k, p += plane) {
      const float4 v = *reinterpret_cast<const float4*>(p);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    return s;
  });
}

template <int B>
void run_rotate(const RotateDims& d, const RowOrder& rows, bool f32, const void* z, const uint16_t* rops, int which,
                void* y, hipStream_t st) {
  const RowLists l{d.T, d.n};
  // Decoded rows, few to an adapter, by 16, others by 64 (us by 16 and by 64
  // rows of 6144 channels, 4 adapters and 64: 512 rows 4.8, 5.4 and 7.0, 9.6;
  // 1024 rows 6.8, 6.9 and 10.6, 11.4; 2048 rows 12.2, 10.6 and 14.1, 14.9)
  const bool few = d.T <= 1024;
  const unsigned tiles = l.cap(few ? LIST_16 : LIST_64);
  if (!few && !f32) {
    const dim3 grid(tiles * ((d.N + 64 * RW - 1) / (64 * RW)));
    const uint16_t* in = static_cast<const uint16_t*>(z);
    uint16_t* out = static_cast<uint16_t*>(y);
    if ((size_t)d.T * d.N * 2 > STREAM_BYTES)
      hipLaunchKernelGGL((rotate_tile_kernel<B, true>), grid, dim3(64 * RW), 0, st, l, rows, in, rops, d.N, which, out);
    else
      hipLaunchKernelGGL((rotate_tile_kernel<B, false>), grid, dim3(64 * RW), 0, st, l, rows, in, rops, d.N, which, out);
    return;
  }
  const dim3 grid(tiles * ((d.N + 127) / 128));
  if (few && f32) hipLaunchKernelGGL((rotate_kernel<16, B, true>), grid, dim3(256), 0, st, l, rows, z, rops, d.N, which, y);
  else if (few) hipLaunchKernelGGL((rotate_kernel<16, B, false>), grid, dim3(256), 0, st, l, rows, z, rops, d.N, which, y);
  else hipLaunchKernelGGL((rotate_kernel<64, B, true>), grid, dim3(256), 0, st, l, rows, z, rops, d.N, which, y);
}

// Pieces of a quarter of few rows, a sixteenth of many: fewer partial sums
// against more workgroups (us, one adapter and 16; 6144 channels: 1024 rows 16,
// 25 by quarters and 19, 32 by sixteenths, 8192 rows 74, 85 and 68, 84; 19456
// channels: 1024 rows 29, 59 and 37, 61, 4096 rows 111, 121 and 108, 122).  A
// step of fp32 rows is longer (1024 rows of 6144 channels, blocks of 16: 22, 25
// and 25, 27; of 2560 channels 20, 17 and 17, 16, 1501 rows 25, 22 and 18, 20).
int sums_list(const RotateDims& d) { return d.T <= (d.f32 ? 1024 : 2048) ? LIST_LONG : LIST_SHORT; }

template <int B>
hipError_t run_sums(const RotateDims& d, const RowOrder& rows, const uint16_t* dy, const void* y, const float* Rf,
                    const uint16_t* rops, uint16_t* dz, float* dq, float* part, hipStream_t st) {
  constexpr int G = 1024 / (B * B);
  const RowLists l{d.T, d.n};
  const int list = sums_list(d);
  const dim3 grid((d.N + SC - 1) / SC, l.cap(list));
  auto sums = [&](auto f32, auto stream) {
    hipLaunchKernelGGL((rotate_sums_kernel<B, decltype(f32)::value, decltype(stream)::value>), grid, dim3(256), 0, st, l,
                       rows, list, dy, y, Rf, rops, d.N, dz, dq, part);
  };
  const bool stream = (size_t)d.T * d.N * 2 > STREAM_BYTES;
  if (d.T > 0) {
    if (d.f32) stream ? sums(std::true_type{}, std::true_type{}) : sums(std::true_type{}, std::false_type{});
    else stream ? sums(std::false_type{}, std::true_type{}) : sums(std::false_type{}, std::false_type{});
  }
  hipLaunchKernelGGL(rotate_join_kernel<B>, dim3((d.N / B + G - 1) / G, d.n), dim3(256), 0, st, l, rows, list, part, Rf,
                     d.N, dq);
  return hipGetLastError();
}

}  // namespace

size_t rotate_ws_bytes(const RotateDims& d, bool bwd) {
  return bwd ? (size_t)RowLists::slots(sums_list(d)) * d.N * 32 * 4 : 0;
}

hipError_t launch_rotate_fwd(const RotateDims& d, const RowOrder& rows, const void* z, const uint16_t* Rops, void* y,
                             hipStream_t st) {
  ProfScope prof(st, "rotate.fwd");
  if (d.b == 32) run_rotate<32>(d, rows, d.f32, z, Rops, 0, y, st);
  else run_rotate<16>(d, rows, d.f32, z, Rops, 0, y, st);
  return hipGetLastError();
}

hipError_t launch_rotate_bwd(const RotateDims& d, const RowOrder& rows, const uint16_t* dy, const void* y,
                             const float* Rf, const uint16_t* Rops, uint16_t* dz, float* dq, char* ws, hipStream_t st) {
  ProfScope prof(st, "rotate.bwd");
  if (dq == nullptr) {
    if (d.b == 32) run_rotate<32>(d, rows, false, dy, Rops, 1, dz, st);
    else run_rotate<16>(d, rows, false, dy, Rops, 1, dz, st);
    return hipGetLastError();
  }
  float* part = reinterpret_cast<float*>(ws);
  return d.b == 32 ? run_sums<32>(d, rows, dy, y, Rf, Rops, dz, dq, part, st)
                   : run_sums<16>(d, rows, dy, y, Rf, Rops, dz, dq, part, st);
}

}  // namespace oft
