// Balance loss of the MoE router with per-expert counts, and its gradient
// (oft_moe_balance, oft_moe_balance_bwd in include/oft.h).
//
// Per sequence of n unmasked tokens, f_e = (pairs routed to e) / (n k) and
// P_e = mean_t p_te:  loss = E sum_e f_e P_e, and with f held fixed
//   d loss / d logit_te = E / n p_te (f_e - sum_j f_j p_tj).
//
// Forward in two launches: workgroups over tiles of tokens leave each tile's
// column sums of p and counts; workgroups over 32 experts of a sequence add
// them in tile order, and the last of a sequence to arrive adds their shares
// of the loss in expert order.  (No float atomics: every sum has one order.)
// The work is one read of the logits, then latency: a softmax per token over
// 16 to 64 lanes with DPP reductions, the next token's row in flight.  Eight
// sequences of 4096 tokens, a quarter of them padding, 384 experts: 13.8 us
// (38 MB) and 6.5 us forward, 20.2 us backward (88 MB, 4.4 TB/s); 512 tokens of
// 64 experts: 3.5, 4.4 and 3.9 us.
#include <math.h>

#include <type_traits>

#include "oft_launch.h"
#include "oft_moe.h"
#include "oft_prof.h"

namespace oft {
namespace {

constexpr int EB = 32;  // experts of a finishing workgroup

// reductions over groups of L lanes, the same bits in each of them; every
// lane of the group is active
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
template <int L, class F>
__device__ __forceinline__ float group_reduce(float v, F f) {
  v = f(v, dpp<0xB1>(v));   // lane ^ 1
  v = f(v, dpp<0x4E>(v));   // lane ^ 2
  v = f(v, dpp<0x141>(v));  // the other four of eight
  v = f(v, dpp<0x140>(v));  // the other eight of sixteen
  if constexpr (L >= 32) v = f(v, __shfl_xor(v, 16));
  if constexpr (L >= 64) v = f(v, __shfl_xor(v, 32));
  return v;
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
  return group_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  return group_reduce<L>(v, [](float a, float b) { return a + b; });
}

// a token's logits: expert sl + L i in register i, -inf past E
template <int L, int NV>
__device__ __forceinline__ void token_row(const float* row, int E, int sl, float (&x)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = sl + L * i < E ? row[sl + L * i] : -INFINITY;
}

// Softmax over a token's lanes: x becomes unnormalised p; returns the
// reciprocal of their sum, 0 for a row of nothing but -inf.  NaN ranks as
// -inf, as in the router.
template <int L, int NV>
__device__ __forceinline__ float token_softmax(float (&x)[NV]) {
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    x[i] = x[i] != x[i] ? -INFINITY : x[i];
    mx = fmaxf(mx, x[i]);
  }
  mx = group_max<L>(mx);
  const float base = mx == -INFINITY ? 0.0f : mx;
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    x[i] = __expf(x[i] - base);
    s += x[i];
  }
  s = group_sum<L>(s);
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
  else if (E <= 384)
    f(integral_constant<int, 64>{}, integral_constant<int, 6>{});
  else if (E <= 512)
    f(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  else
    f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

// Tiles of a forward call and where their parts lie in the workspace:
// [S tiles] rows of E column sums and E counts, a token count per tile, a
// share of the loss per finishing workgroup, an arrival counter per sequence.
struct Plan {
  int S, tile, tiles, eb;  // sequences, tokens of a tile, tiles and finishing workgroups of a sequence
  size_t p, c, used, share, arrived, bytes;
};
Plan plan_of(const MoeDims& d, int seq_len) {
  Plan q;
  q.S = d.T / seq_len;
  // about a thousand workgroups, so that each SIMD has waves to overlap; a
  // tile's sums cost E (4 + 2) bytes written and read again beside its 4 E
  // bytes per token
  q.tile = d.T <= 8192 ? 16 : d.T <= 32768 ? 32 : 64;
  q.tiles = (seq_len + q.tile - 1) / q.tile;
  q.eb = (d.E + EB - 1) / EB;
  const size_t n = (size_t)q.S * q.tiles;
  size_t off = 0;
  const auto take = [&](size_t bytes) {
    const size_t at = off;
    off += (bytes + 255) & ~(size_t)255;
    return at;
  };
  q.p = take(n * d.E * 4);
  q.c = take(n * d.E * 2);
  q.used = take(n * 4);
  q.share = take((size_t)q.S * q.eb * 4);
  q.arrived = take((size_t)q.S * 4);
  q.bytes = off;
  return q;
}

struct Parts {
  float* p;
  uint16_t* c;  // at most 64 tokens of 16 pairs
  int* used;
  float* share;
  int* arrived;
};

template <int L, int NV>
__global__ __launch_bounds__(256) void balance_tile_kernel(MoeBalancePtrs q, Parts w, int E, int k, int seq_len,
                                                           int tile, int tiles) {
  constexpr int TPW = 64 / L, TPB = 4 * TPW;  // tokens at a time of a wave, of the workgroup
  __shared__ float col[4][L * NV];
  __shared__ int cnt[L * NV];
  __shared__ int used;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, sl = lane % L;
  const int seq = blockIdx.x / tiles, at = blockIdx.x % tiles;
  const size_t first = (size_t)seq * seq_len;
  const int t1 = min(seq_len, (at + 1) * tile);
  for (int e = tid; e < L * NV; e += 256) cnt[e] = 0;
  if (tid == 0) {
    used = 0;
    if (at == 0) w.arrived[seq] = 0;  // for the finishing launch
  }
  __syncthreads();
  float acc[NV], x[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) acc[i] = 0.0f;
  int t = at * tile + wave * TPW + lane / L;
  const auto valid = [&](int u) { return u < t1 && !(q.mask && q.mask[first + u] == 0); };
  bool ok = valid(t);
  int e = -1;
  if (ok) {
    token_row<L, NV>(q.logits + (first + t) * E, E, sl, x);
    if (sl < k) e = q.topk_idx[(first + t) * k + sl];
  }
  while (t < t1) {  // (whole groups of lanes agree on t, ok and next: the reductions stay inside a group)
    const int tn = t + TPB;
    const bool next = valid(tn);
    float y[NV];
    int en = -1;
    if (next) {
      token_row<L, NV>(q.logits + (first + tn) * E, E, sl, y);
      if (sl < k) en = q.topk_idx[(first + tn) * k + sl];
    }
    if (ok) {
      const float r = token_softmax<L, NV>(x);
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] = fmaf(x[i], r, acc[i]);
      if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
      if (sl == 0) atomicAdd(&used, 1);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = y[i];
    e = en;
    ok = next;
    t = tn;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int off = 32; off >= L; off >>= 1) acc[i] += __shfl_xor(acc[i], off);
    if (lane < L) col[wave][sl + L * i] = acc[i];
  }
  __syncthreads();
  const size_t out = (size_t)blockIdx.x * E;
  for (int i = tid; i < E; i += 256) {
    w.p[out + i] = (col[0][i] + col[1][i]) + (col[2][i] + col[3][i]);
    w.c[out + i] = (uint16_t)cnt[i];
  }
  if (tid == 0) w.used[blockIdx.x] = used;
}

// Experts [EB b, EB (b + 1)) of a sequence: eight threads each, every eighth
// tile.  (Sequences along x, experts along y: a million sequences of one token
// times 1024 experts are more threads than one grid dimension takes.)
__global__ __launch_bounds__(256) void balance_finish_kernel(MoeBalancePtrs q, Parts w, int E, int k, int tiles,
                                                             int eb) {
  __shared__ float sp[8][EB];
  __shared__ int sc[8][EB], sn[4], last;
  const int seq = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int i = tid % EB, g = tid / EB, e = b * EB + i;
  const size_t row = (size_t)seq * tiles;
  int n = 0;
  for (int t = tid; t < tiles; t += 256) n += w.used[row + t];
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) n += __shfl_xor(n, off);
  if ((tid & 63) == 0) sn[tid >> 6] = n;
  float p = 0.0f;
  int c = 0;
  if (e < E) {
#pragma unroll 8
    for (int t = g; t < tiles; t += 8) {
      p += w.p[(row + t) * E + e];
      c += w.c[(row + t) * E + e];
    }
  }
  sp[g][i] = p;
  sc[g][i] = c;
  __syncthreads();
  n = sn[0] + sn[1] + sn[2] + sn[3];
  const float invn = n > 0 ? 1.0f / (float)n : 0.0f;
  if (tid < 64) {  // (the whole first wave: its upper half adds zeros)
    float mean = 0.0f;
    if (tid < EB && e < E) {
      p = 0.0f;
      c = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p += sp[j][i];
        c += sc[j][i];
      }
      mean = p * invn;
      q.counts[(size_t)seq * E + e] = c;
      if (q.mean_prob) q.mean_prob[(size_t)seq * E + e] = mean;
      mean *= (float)c;
    }
    const float share = group_sum<64>(mean);
    if (tid == 0) {
      // device scope: the workgroups of a sequence may sit on different dies
      __hip_atomic_store(&w.share[(size_t)seq * eb + b], share, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = __hip_atomic_fetch_add(&w.arrived[seq], 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == eb - 1;
    }
  }
  __syncthreads();
  if (last && tid == 0) {
    float sum = 0.0f;
    for (int j = 0; j < eb; ++j)
      sum += __hip_atomic_load(&w.share[(size_t)seq * eb + j], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    q.tokens[seq] = n;
    q.loss[seq] = sum * invn * ((float)E / (float)k);
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
  float p[NV], c[NV];
  token_row<L, NV>(logits + (size_t)t * E, E, sl, p);
#pragma unroll
  for (int i = 0; i < NV; ++i) c[i] = sl + L * i < E ? (float)counts[(size_t)seq * E + sl + L * i] : 0.0f;
  const float invn = 1.0f / (float)tokens[seq];
  const float scale = g_loss[seq] * (float)E * invn * invn / (float)k;
  const float r = token_softmax<L, NV>(p);
  float dot = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    p[i] *= r;
    dot = fmaf(c[i], p[i], dot);
  }
  dot = group_sum<L>(dot);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = sl + L * i;
    if (e < E) {
      const float v = scale * p[i] * (c[i] - dot);
      out[e] = accumulate ? out[e] + v : v;
    }
  }
}

}  // namespace

size_t moe_balance_ws_bytes(const MoeDims& d, int seq_len) { return plan_of(d, seq_len).bytes; }

hipError_t launch_moe_balance(const MoeDims& d, int seq_len, const MoeBalancePtrs& q, char* ws, hipStream_t st) {
  ProfScope prof(st, "moe.balance");
  const Plan s = plan_of(d, seq_len);
  const Parts w{reinterpret_cast<float*>(ws + s.p), reinterpret_cast<uint16_t*>(ws + s.c),
                reinterpret_cast<int*>(ws + s.used), reinterpret_cast<float*>(ws + s.share),
                reinterpret_cast<int*>(ws + s.arrived)};
  lane_shape(d.E, [&](auto l, auto nv) {
    constexpr int Lc = decltype(l)::value, NVc = decltype(nv)::value;
    hipLaunchKernelGGL((balance_tile_kernel<Lc, NVc>), dim3((size_t)s.S * s.tiles), dim3(256), 0, st, q, w, d.E, d.k,
                       seq_len, s.tile, s.tiles);
  });
  hipLaunchKernelGGL(balance_finish_kernel, dim3(s.S, s.eb), dim3(256), 0, st, q, w, d.E, d.k, s.tiles, s.eb);
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
