// Balance loss of the MoE router with per-expert counts, and its gradient
// (oft_moe_balance, oft_moe_balance_bwd in include/oft.h).
//
// Per sequence of n unmasked tokens, f_e = (pairs routed to e) / (n k) and
// P_e = mean_t p_te:  loss = E sum_e f_e P_e, and with f held fixed
//   d loss / d logit_te = E / n p_te (f_e - sum_j f_j p_tj).
//
// Forward in two launches: workgroups over tiles of tokens leave each tile's
// column sums of p and counts, then one workgroup per sequence adds them in
// tile order (no float atomics: the sums have one order).
#include <math.h>

#include <type_traits>

#include "oft_launch.h"
#include "oft_moe.h"
#include "oft_prof.h"

namespace oft {
namespace {

constexpr int TILE = 64;  // tokens of a forward workgroup

// Softmax of a token's row over its group of L lanes (NV experts per lane,
// expert sl + L i): unnormalised p[i] and the reciprocal of their sum, 0 for
// a row of nothing but -inf.  NaN ranks as -inf, as in the router.
template <int L, int NV>
__device__ __forceinline__ float token_softmax(const float* row, int E, int sl, float (&p)[NV]) {
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = sl + L * i;
    const float x = e < E ? row[e] : -INFINITY;
    p[i] = x != x ? -INFINITY : x;
    mx = fmaxf(mx, p[i]);
  }
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
  const float base = mx == -INFINITY ? 0.0f : mx;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    p[i] = __expf(p[i] - base);
    s += p[i];
  }
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) s += __shfl_xor(s, off);
  return s == 0.0f ? 0.0f : 1.0f / s;
}

// f(L, NV) for E experts: L lanes per token, NV experts per lane
template <class F>
void lane_shape(int E, F&& f) {
  using std::integral_constant;
  if (E <= 64)
    f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  else if (E <= 128)
    f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  else if (E <= 256)
    f(integral_constant<int, 32>{}, integral_constant<int, 8>{});
  else if (E <= 512)
    f(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  else
    f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

template <int L, int NV>
__global__ __launch_bounds__(256) void balance_tile_kernel(MoeBalancePtrs q, int E, int k, int seq_len,
                                                           int tiles, float* __restrict__ part_p, int* __restrict__ part_c) {
  constexpr int TPW = 64 / L, TPB = 4 * TPW;  // tokens of a wave, of the workgroup
  __shared__ float col[4][L * NV];
  __shared__ int cnt[L * NV];
  __shared__ int used;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, sl = lane % L;
  const int seq = blockIdx.x / tiles, tile = blockIdx.x % tiles;
  const int t0 = tile * TILE, t1 = min(seq_len, t0 + TILE);
  const size_t first = (size_t)seq * seq_len;
  for (int e = tid; e < L * NV; e += 256) cnt[e] = 0;
  if (tid == 0) used = 0;
  __syncthreads();
  float acc[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) acc[i] = 0.0f;
  for (int t = t0 + wave * TPW + lane / L; t < t1; t += TPB) {
    if (q.mask && q.mask[first + t] == 0) continue;  // whole groups: the shuffles stay inside a group
    float p[NV];
    const float r = token_softmax<L, NV>(q.logits + (first + t) * E, E, sl, p);
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] = fmaf(p[i], r, acc[i]);
    if (sl < k) {
      const int e = q.topk_idx[(first + t) * k + sl];
      if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
    }
    if (sl == 0) atomicAdd(&used, 1);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int off = 32; off >= L; off >>= 1) acc[i] += __shfl_xor(acc[i], off);
    if (lane < L) col[wave][sl + L * i] = acc[i];
  }
  __syncthreads();
  const size_t at = (size_t)blockIdx.x * (E + 1);
  for (int e = tid; e < E; e += 256) {
    part_p[at + e] = (col[0][e] + col[1][e]) + (col[2][e] + col[3][e]);
    part_c[at + e] = cnt[e];
  }
  if (tid == 0) part_c[at + E] = used;
}

__global__ __launch_bounds__(256) void balance_finish_kernel(MoeBalancePtrs q, int E, int k, int tiles,
                                                             const float* __restrict__ part_p,
                                                             const int* __restrict__ part_c) {
  __shared__ float sh[4];
  const int seq = blockIdx.x, tid = threadIdx.x;
  const size_t at = (size_t)seq * tiles * (E + 1);
  int n = 0;
  for (int i = 0; i < tiles; ++i) n += part_c[at + (size_t)i * (E + 1) + E];
  const float invn = n > 0 ? 1.0f / (float)n : 0.0f;
  float sum = 0.0f;
  for (int e = tid; e < E; e += 256) {
    float p = 0.0f;
    int c = 0;
    for (int i = 0; i < tiles; ++i) {
      p += part_p[at + (size_t)i * (E + 1) + e];
      c += part_c[at + (size_t)i * (E + 1) + e];
    }
    q.counts[(size_t)seq * E + e] = c;
    if (q.mean_prob) q.mean_prob[(size_t)seq * E + e] = p * invn;
    sum = fmaf((float)c, p * invn, sum);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
  if ((tid & 63) == 0) sh[tid >> 6] = sum;
  __syncthreads();
  if (tid == 0) {
    q.tokens[seq] = n;
    q.loss[seq] = ((sh[0] + sh[1]) + (sh[2] + sh[3])) * invn * ((float)E / (float)k);
  }
}

template <int L, int NV>
__global__ __launch_bounds__(256) void balance_bwd_kernel(const float* __restrict__ logits,
                                                          const uint8_t* __restrict__ mask,
                                                          const int* __restrict__ counts,
                                                          const int* __restrict__ tokens,
                                                          const float* __restrict__ g_loss, int T, int E, int k,
                                                          int seq_len, int accumulate, float* __restrict__ dl) {
  constexpr int TPW = 64 / L;
  const int lane = threadIdx.x & 63, sl = lane % L;
  const int t = (blockIdx.x * 4 + (threadIdx.x >> 6)) * TPW + lane / L;
  if (t >= T) return;  // whole groups leave together
  float* out = dl + (size_t)t * E;
  if (mask && mask[t] == 0) {
    if (!accumulate) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (sl + L * i < E) out[sl + L * i] = 0.0f;
    }
    return;
  }
  const int seq = t / seq_len;
  const float invn = 1.0f / (float)tokens[seq];
  const float scale = g_loss[seq] * (float)E * invn * invn / (float)k;
  float p[NV], c[NV];
  const float r = token_softmax<L, NV>(logits + (size_t)t * E, E, sl, p);
  float dot = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = sl + L * i;
    c[i] = e < E ? (float)counts[(size_t)seq * E + e] : 0.0f;
    p[i] *= r;
    dot = fmaf(c[i], p[i], dot);
  }
#pragma unroll
  for (int off = L / 2; off >= 1; off >>= 1) dot += __shfl_xor(dot, off);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = sl + L * i;
    if (e < E) {
      const float v = scale * p[i] * (c[i] - dot);
      out[e] = accumulate ? out[e] + v : v;
    }
  }
}

int tiles_of(int seq_len) { return (seq_len + TILE - 1) / TILE; }

}  // namespace

size_t moe_balance_ws_bytes(const MoeDims& d, int seq_len) {
  const size_t parts = (size_t)(d.T / seq_len) * tiles_of(seq_len) * (d.E + 1);
  return ((parts * 4 + 255) & ~(size_t)255) * 2;
}

hipError_t launch_moe_balance(const MoeDims& d, int seq_len, const MoeBalancePtrs& q, char* ws, hipStream_t st) {
  ProfScope prof(st, "moe.balance");
  const int S = d.T / seq_len, tiles = tiles_of(seq_len);
  float* part_p = reinterpret_cast<float*>(ws);
  int* part_c = reinterpret_cast<int*>(ws + moe_balance_ws_bytes(d, seq_len) / 2);
  lane_shape(d.E, [&](auto l, auto nv) {
    constexpr int Lc = decltype(l)::value, NVc = decltype(nv)::value;
    hipLaunchKernelGGL((balance_tile_kernel<Lc, NVc>), dim3((size_t)S * tiles), dim3(256), 0, st, q, d.E, d.k, seq_len,
                       tiles, part_p, part_c);
  });
  hipLaunchKernelGGL(balance_finish_kernel, dim3(S), dim3(256), 0, st, q, d.E, d.k, tiles, part_p, part_c);
  return hipGetLastError();
}

hipError_t launch_moe_balance_bwd(const MoeDims& d, int seq_len, const float* logits, const uint8_t* mask,
                                  const int* counts, const int* tokens, const float* g_loss, float* d_logits,
                                  bool accumulate, hipStream_t st) {
  ProfScope prof(st, "moe.balance_bwd");
  lane_shape(d.E, [&](auto l, auto nv) {
    constexpr int Lc = decltype(l)::value, NVc = decltype(nv)::value;
    const int per = 4 * (64 / Lc);  // tokens per workgroup
    hipLaunchKernelGGL((balance_bwd_kernel<Lc, NVc>), dim3((d.T + per - 1) / per), dim3(256), 0, st, logits, mask,
                       counts, tokens, g_loss, d.T, d.E, d.k, seq_len, accumulate ? 1 : 0, d_logits);
  });
  return hipGetLastError();
}

}  // namespace oft
