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
// its result, 16 consecutive ones of a row.
//
// fp32 rows are split into three bf16 parts whose sum is the value; bf16 rows
// and rotations are operands as they are.
#include "adapter_device.h"
#include "gemm_nn.h"
#include "oft_prof.h"

namespace oft {
namespace {

// Rotation operand of channels n0 .. n0 + 31 (pack `which`: 0 R, 1 R^T):
// operand row l32 is channel 16 (l32 / 4 % 2) + 4 (l32 / 8) + l32 % 4, whose
// results are then registers 0 .. 15 of lane group l32 / 4 % 2; contraction
// item p of step t in lane group g is channel 16 g + 8 t + p.
template <int B>
__device__ __forceinline__ void load_rotation(const uint16_t* __restrict__ rops, int n0, int which, int l32, int g,
                                              uint4 (&o)[2]) {
  const int gr = (l32 >> 2) & 1, c = 4 * (l32 >> 3) + (l32 & 3);  // channel 16 gr + c
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    if constexpr (B == 32) {
      o[t] = *reinterpret_cast<const uint4*>(rops + (size_t)(n0 / 32) * 2048 + which * 1024 + (16 * gr + c) * 32 +
                                             16 * g + 8 * t);
    } else {
      o[t] = gr == g ? *reinterpret_cast<const uint4*>(rops + (size_t)(n0 / 16 + g) * 512 + which * 256 + c * 16 + 8 * t)
                     : zero4();
    }
  }
}

template <bool F32>
__device__ __forceinline__ f32x16 rotate(const uint4 (&rot)[2], const Oct<F32> (&z)[2]) {
  constexpr int P = Oct<F32>::P;
  f32x16 o;
#pragma unroll
  for (int r = 0; r < 16; ++r) o[r] = 0.0f;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    uint4 p[P];
    z[t].parts(p);
#pragma unroll
    for (int k = P - 1; k >= 0; --k) o = mfma32(as_bf16x8(rot[t]), as_bf16x8(p[k]), o);
  }
  return o;
}

template <bool F32>
__device__ __forceinline__ void store16(void* out, size_t at, const f32x16& o) {
  if constexpr (F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  } else {
    uint4* q = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      q[i] = make_uint4(pack_bf16x2(o[8 * i], o[8 * i + 1]), pack_bf16x2(o[8 * i + 2], o[8 * i + 3]),
                        pack_bf16x2(o[8 * i + 4], o[8 * i + 5]), pack_bf16x2(o[8 * i + 6], o[8 * i + 7]));
  }
}

template <bool F32>
__device__ __forceinline__ void copy16(void* out, size_t at, const Oct<F32> (&z)[2]) {
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    if constexpr (F32) {
      float4* q = reinterpret_cast<float4*>(static_cast<float*>(out) + at + 8 * t);
      q[0] = z[t].a;
      q[1] = z[t].b;
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at + 8 * t) = z[t].u;
    }
  }
}

// ------------------------------------------------------------------ rows
template <int TM, int B, bool F32>
__global__ __launch_bounds__(256) void rotate_kernel(RowLists l, RowOrder rows, const void* z,
                                                     const uint16_t* __restrict__ rops, int N, int which, void* y) {
  constexpr int XG = (TM + 31) / 32;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l32 = lane & 31, g = lane >> 5;
  const int wgs = (N + 127) / 128;
  const int tile = blockIdx.x / wgs, n0 = (blockIdx.x % wgs) * 128 + 32 * wave;
  int4 e;
  if (n0 >= N || !list_entry(l, rows.tiles, TM == 16 ? LIST_16 : LIST_64, tile, e)) return;
  Oct<F32> x[XG][2];
  size_t at[XG];
#pragma unroll
  for (int i = 0; i < XG; ++i) {
    at[i] = (size_t)row_at(l, rows.order, e.y + min(32 * i + l32, e.z - 1)) * N + n0 + 16 * g;
#pragma unroll
    for (int t = 0; t < 2; ++t) x[i][t].load(z, at[i] + 8 * t);
  }
  if (e.x < 0) {
    if (y == z) return;
#pragma unroll
    for (int i = 0; i < XG; ++i)
      if (32 * i + l32 < e.z) copy16<F32>(y, at[i], x[i]);
    return;
  }
  uint4 rot[2];
  load_rotation<B>(rops + (size_t)e.x * N * B * 2, n0, which, l32, g, rot);
#pragma unroll
  for (int i = 0; i < XG; ++i) {
    const f32x16 o = rotate<F32>(rot, x[i]);
    if (32 * i + l32 < e.z) store16<F32>(y, at[i], o);
  }
}

// ------------------------------------------------------- sums over the rows
// One piece of an adapter's rows and 128 channels: dz of every row (dz may be
// NULL), S of the channels' blocks.  Tiles of 32 rows go to LDS in row order;
// S's operands, which run along the rows, are read with the transposing load.
constexpr int SC = 128, SR = 32, LDS_ROW = SC + 16;

template <int B, bool F32>
__global__ __launch_bounds__(256) void rotate_sums_kernel(RowLists l, RowOrder rows, int list,
                                                          const uint16_t* __restrict__ dy, const void* __restrict__ y,
                                                          const float* __restrict__ Rf,
                                                          const uint16_t* __restrict__ rops, int N, uint16_t* dz,
                                                          float* __restrict__ dq, float* __restrict__ part) {
  constexpr int P = Oct<F32>::P, G = 1024 / (B * B), NP = B * (B - 1) / 2;
  constexpr int TILE = SR * LDS_ROW;
  constexpr int GRAD = 3 * G * B * (B + 4);                          // floats of the Cayley gradient
  constexpr int FLOATS = (1 + P) * TILE / 2 > 4 * 32 * 36 + GRAD ? (1 + P) * TILE / 2 : 4 * 32 * 36 + GRAD;
  __shared__ __attribute__((aligned(16))) float lds[FLOATS];
  uint16_t* ds = reinterpret_cast<uint16_t*>(lds);
  uint16_t* ys = ds + TILE;

  int4 e;
  if (!list_entry(l, rows.tiles, list, blockIdx.y, e)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int l32 = lane & 31, l16 = lane & 15, g = lane >> 5;
  const int n0 = blockIdx.x * SC, nw = n0 + 32 * wave;
  const bool w_ok = nw < N;
  // thread: 8 channels of rows tid / 16 and tid / 16 + 16
  const int c = n0 + 8 * (tid & 15), r = tid >> 4;
  const bool c_ok = c < N;

  if (e.x < 0) {  // rows of the base model: dz = dy, no sums
    if (dz == nullptr || !c_ok || dz == dy) return;
    for (int i = r; i < e.z; i += 16) {
      const size_t at = (size_t)row_at(l, rows.order, e.y + i) * N + c;
      *reinterpret_cast<uint4*>(dz + at) = *reinterpret_cast<const uint4*>(dy + at);
    }
    return;
  }
  uint4 rot[2] = {zero4(), zero4()};
  if (dz != nullptr && w_ok) load_rotation<B>(rops + (size_t)e.x * N * B * 2, nw, 1, l32, g, rot);

  f32x16 acc;
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
  Oct<false> d[2];
  Oct<F32> v[2];
  auto load = [&](int r0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int k = r0 + r + 16 * i;
      if (k < e.z && c_ok) {
        const size_t at = (size_t)row_at(l, rows.order, e.y + k) * N + c;
        d[i].load(dy, at);
        v[i].load(y, at);
      } else {
        d[i].zero();
        v[i].zero();
      }
    }
  };
  load(0);
  for (int r0 = 0; r0 < e.z; r0 += SR) {
    __syncthreads();  // the last step's reads are done
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = (r + 16 * i) * LDS_ROW + 8 * (tid & 15);
      *reinterpret_cast<uint4*>(ds + at) = d[i].u;
      uint4 p[P];
      v[i].parts(p);
#pragma unroll
      for (int k = 0; k < P; ++k) *reinterpret_cast<uint4*>(ys + k * TILE + at) = p[k];
    }
    __syncthreads();
    if (r0 + SR < e.z) load(r0 + SR);
    if (dz != nullptr) {
      Oct<false> x[2];
#pragma unroll
      for (int t = 0; t < 2; ++t)
        x[t].u = *reinterpret_cast<const uint4*>(ds + l32 * LDS_ROW + 32 * wave + 16 * g + 8 * t);
      const f32x16 o = rotate<false>(rot, x);
      if (w_ok && r0 + l32 < e.z)
        store16<false>(dz, (size_t)row_at(l, rows.order, e.y + r0 + l32) * N + nw + 16 * g, o);
    }
    // lane l16 of a 16-lane group: 8 rows of one of its 16 channels
#pragma unroll
    for (int k0 = 0; k0 < SR; k0 += 16) {
      const int at = (k0 + 8 * g + (l16 >> 2)) * LDS_ROW + 32 * wave + 16 * ((lane >> 4) & 1) + 4 * (l16 & 3);
      const uint2 dl = nn::ds_read_tr16(ds + at), dh = nn::ds_read_tr16(ds + at + 4 * LDS_ROW);
      const bf16x8 a = as_bf16x8(make_uint4(dl.x, dl.y, dh.x, dh.y));
#pragma unroll
      for (int k = P - 1; k >= 0; --k) {
        const uint16_t* q = ys + k * TILE + at;
        const uint2 lo = nn::ds_read_tr16(q), hi = nn::ds_read_tr16(q + 4 * LDS_ROW);
        acc = mfma32(a, as_bf16x8(make_uint4(lo.x, lo.y, hi.x, hi.y)), acc);
      }
    }
  }
  // lane: column l32 of S, rows 8 (i / 4) + 4 g + i % 4
  if (e.w >= 0) {
    if (!w_ok) return;
    float* out = part + ((size_t)min(e.w, RowLists::slots(list) - 1) * (N / 32) + nw / 32) * 1024;
#pragma unroll
    for (int i = 0; i < 16; ++i) out[(8 * (i / 4) + 4 * g + i % 4) * 32 + l32] = acc[i];
    return;
  }
  __syncthreads();
  float* S = lds;  // [4][32][36]
#pragma unroll
  for (int i = 0; i < 16; ++i) S[(wave * 32 + 8 * (i / 4) + 4 * g + i % 4) * 36 + l32] = acc[i];
  const float* R = Rf + (size_t)e.x * N * B;
  float* out = dq + (size_t)e.x * (N / B) * NP;
  for (int h = 0; h < 4 * 32 / (G * B); ++h) {  // G blocks at a time
    const int b0 = n0 / B + h * G, nb = min(G, N / B - b0);
    if (nb <= 0) break;
    __syncthreads();
    cayley_grad_group<B>(lds + 4 * 32 * 36, R + (size_t)b0 * B * B, out + (size_t)b0 * NP, nb, tid,
                         [&](int gb, int rr, int cc) {
                           const int ch = (h * G + gb) * B;  // channel within the 128
                           return *reinterpret_cast<const float4*>(S + (ch + rr) * 36 + (ch & 31) + cc);
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
  const int first = rows.tiles[l.part_at(list) + ad];
  const int slots = min(pieces, RowLists::slots(list) - first);
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
  // decoded rows: few to an adapter
  const bool few = d.T <= 1024;
  const dim3 grid((unsigned)l.cap(few ? LIST_16 : LIST_64) * ((d.N + 127) / 128));
  if (few) {
    if (f32) hipLaunchKernelGGL((rotate_kernel<16, B, true>), grid, dim3(256), 0, st, l, rows, z, rops, d.N, which, y);
    else hipLaunchKernelGGL((rotate_kernel<16, B, false>), grid, dim3(256), 0, st, l, rows, z, rops, d.N, which, y);
  } else {
    if (f32) hipLaunchKernelGGL((rotate_kernel<64, B, true>), grid, dim3(256), 0, st, l, rows, z, rops, d.N, which, y);
    else hipLaunchKernelGGL((rotate_kernel<64, B, false>), grid, dim3(256), 0, st, l, rows, z, rops, d.N, which, y);
  }
}

int sums_list(const RotateDims& d) { return (d.N + SC - 1) / SC >= 128 ? LIST_LONG : LIST_SHORT; }

template <int B>
hipError_t run_sums(const RotateDims& d, const RowOrder& rows, const uint16_t* dy, const void* y, const float* Rf,
                    const uint16_t* rops, uint16_t* dz, float* dq, float* part, hipStream_t st) {
  constexpr int G = 1024 / (B * B);
  const RowLists l{d.T, d.n};
  const int list = sums_list(d);
  const dim3 grid((d.N + SC - 1) / SC, l.cap(list));
  if (d.T == 0) {
  } else if (d.f32)
    hipLaunchKernelGGL((rotate_sums_kernel<B, true>), grid, dim3(256), 0, st, l, rows, list, dy, y, Rf, rops, d.N, dz, dq,
                       part);
  else
    hipLaunchKernelGGL((rotate_sums_kernel<B, false>), grid, dim3(256), 0, st, l, rows, list, dy, y, Rf, rops, d.N, dz,
                       dq, part);
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
