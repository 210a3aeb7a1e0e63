// Losses on vocabulary logits (include/oft.h): log-probabilities of given
// tokens with entropy and top alternatives, distillation from a teacher's
// top logits, and their gradients.  One workgroup of 256 threads per row.
#include <math.h>

#include "oft_device.h"
#include "oft_launch.h"
#include "oft_prof.h"
#include "oft_vocab.h"

namespace oft {
namespace {

constexpr float LOG2E = 1.44269504088896340736f;
// below this a log-probability has p = 0 in fp32; the clamp keeps 0 * z finite
constexpr float LOWEST = -128.0f;

template <class E>
__device__ __forceinline__ float to_f32(E v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) {
  return bf16_to_f32(v);
}
template <class E>
__device__ __forceinline__ E from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) {
  return (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
}

// order of the top alternatives: larger value, then lower column; NaN ranks
// as -inf
__device__ __forceinline__ bool beats(float v, int i, float w, int j) { return v > w || (v == w && i < j); }

// sum (or maximum) over the 256 threads, the same value in every thread
__device__ float block_sum(float v, float* sh) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  return (sh[0] + sh[1]) + (sh[2] + sh[3]);
}
__device__ float block_max(float v, float* sh) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = fmaxf(v, __shfl_xor(v, off));
  __syncthreads();
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  return fmaxf(fmaxf(sh[0], sh[1]), fmaxf(sh[2], sh[3]));
}

// m, l and sum e^z z / s of a row
template <class E>
__device__ void row_stats(const E* row, int V, float invtau, float* sh, float& m, float& l, float& wz) {
  float mx = -INFINITY;
  for (int i = threadIdx.x; i < V; i += 256) mx = fmaxf(mx, to_f32<E>(row[i]));
  m = block_max(mx, sh);
  const float base = m == -INFINITY ? 0.0f : m;
  float s = 0.0f, w = 0.0f;
  for (int i = threadIdx.x; i < V; i += 256) {
    const float z = (to_f32<E>(row[i]) - base) * invtau;
    const float e = __expf(z);
    s += e;
    w = fmaf(e, fmaxf(z, LOWEST), w);
  }
  s = block_sum(s, sh);
  w = block_sum(w, sh);
  l = __logf(s);  // -inf for an empty row
  wz = s > 0.0f ? w / s : 0.0f;
  if (s != s) wz = s;
}

template <class E>
__global__ __launch_bounds__(256) void logprobs_kernel(VocabDims d, LogprobPtrs q) {
  __shared__ float sh[4];
  __shared__ float sv[4];
  __shared__ int si[4];
  const int t = blockIdx.x, tid = threadIdx.x;
  const E* row = static_cast<const E*>(q.logits) + (size_t)t * d.ld;
  float m, l, wz;
  row_stats<E>(row, d.V, d.invtau, sh, m, l, wz);
  if (tid == 0) {
    q.stats[2 * (size_t)t] = m;
    q.stats[2 * (size_t)t + 1] = l;
    if (q.entropy) q.entropy[t] = l == -INFINITY ? 0.0f : l - wz;
    if (q.logp) {
      const int lab = q.labels[t];
      float lp = NAN;
      if (lab == -1) lp = 0.0f;
      else if (lab >= 0 && lab < d.V) lp = l == -INFINITY ? -INFINITY : (to_f32<E>(row[lab]) - m) * d.invtau - l;
      q.logp[t] = lp;
    }
  }
  // slot j: the best column after the last one found
  float pv = INFINITY;
  int pi = -1;
  for (int j = 0; j < d.k; ++j) {
    float bv = -INFINITY;
    int bi = 0x7fffffff;
    for (int i = tid; i < d.V; i += 256) {
      float x = to_f32<E>(row[i]);
      if (x != x) x = -INFINITY;
      if ((j == 0 || beats(pv, pi, x, i)) && beats(x, i, bv, bi)) {
        bv = x;
        bi = i;
      }
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const float ov = __shfl_xor(bv, off);
      const int oi = __shfl_xor(bi, off);
      if (beats(ov, oi, bv, bi)) {
        bv = ov;
        bi = oi;
      }
    }
    __syncthreads();
    if ((tid & 63) == 0) {
      sv[tid >> 6] = bv;
      si[tid >> 6] = bi;
    }
    __syncthreads();
    bv = sv[0];
    bi = si[0];
    for (int w = 1; w < 4; ++w)
      if (beats(sv[w], si[w], bv, bi)) {
        bv = sv[w];
        bi = si[w];
      }
    if (tid == 0) {
      q.top_idx[(size_t)t * d.k + j] = bi;
      const float lp = l == -INFINITY ? -INFINITY : (bv - m) * d.invtau - l;
      q.top_logp[(size_t)t * d.k + j] = l != l ? NAN : lp;
    }
    pv = bv;
    pi = bi;
  }
}

template <class E>
__global__ __launch_bounds__(256) void logprobs_bwd_kernel(VocabDims d, LogprobGradPtrs q) {
  const int t = blockIdx.x;
  const E* row = static_cast<const E*>(q.logits) + (size_t)t * d.ld;
  E* out = static_cast<E*>(q.d_logits) + (size_t)t * d.ldg;
  const float m = q.stats[2 * (size_t)t], l = q.stats[2 * (size_t)t + 1];
  const int lab = q.labels ? q.labels[t] : -1;
  float gl = lab == -1 ? 0.0f : q.g_logp[t];
  const float ge = q.g_entropy ? q.g_entropy[t] : 0.0f;
  const float H = ge != 0.0f ? q.entropy[t] : 0.0f;
  // nothing to do, or a label that names no column
  const bool zero = gl == 0.0f && ge == 0.0f;
  const bool bad = !zero && (lab < -1 || lab >= d.V);
  const bool none = zero || bad || l == -INFINITY;
  for (int i = threadIdx.x; i < d.V; i += 256) {
    float v = bad ? NAN : 0.0f;
    if (!none) {
      const float lp = (to_f32<E>(row[i]) - m) * d.invtau - l;
      v = -__expf(lp) * (gl + ge * (fmaxf(lp, LOWEST) + H));
      if (i == lab) v += gl;
      v *= d.invtau;
    }
    if (d.accumulate) v += to_f32<E>(out[i]);
    out[i] = from_f32<E>(v);
  }
}

// the teacher's row: thread j < k holds entry j; q of the row (0 for an
// entry without weight), its log, and whether the row has any weight; q is
// NaN throughout if an entry is out of range, NaN or +inf
__device__ void teacher_row(const VocabDims& d, int t, const int* idx, const float* teacher, float* sh, int& ix,
                            float& qj, float& logq, bool& any) {
  const int tid = threadIdx.x;
  float v = -INFINITY, bad = 0.0f;
  ix = -1;
  if (tid < d.k) {
    ix = idx[(size_t)t * d.k + tid];
    if (ix != -1) v = teacher[(size_t)t * d.k + tid];
    if (ix < -1 || ix >= d.V || v != v || v == INFINITY) {
      bad = 1.0f;
      v = 0.0f;
      ix = -1;
    }
  }
  const bool nan = block_max(bad, sh) != 0.0f;
  const float m = block_max(v, sh);
  any = m != -INFINITY;
  const float z = any ? (v - m) * d.invtau : -INFINITY;
  const float e = __expf(z);
  const float s = block_sum(e, sh);
  qj = nan ? NAN : any ? e / s : 0.0f;
  logq = z - __logf(s);
}

template <class E>
__global__ __launch_bounds__(256) void distill_kernel(VocabDims d, const void* logits, const int* idx,
                                                      const float* teacher, float* loss, float* stats) {
  __shared__ float sh[4];
  const int t = blockIdx.x;
  const E* row = static_cast<const E*>(logits) + (size_t)t * d.ld;
  float m, l, wz;
  row_stats<E>(row, d.V, d.invtau, sh, m, l, wz);
  int ix;
  float qj, logq;
  bool any;
  teacher_row(d, t, idx, teacher, sh, ix, qj, logq, any);
  float c = 0.0f;
  if (qj != qj) c = NAN;
  else if (qj > 0.0f) {
    const float lp = l == -INFINITY ? -INFINITY : (to_f32<E>(row[ix]) - m) * d.invtau - l;
    c = qj * (logq - lp);
  }
  c = block_sum(c, sh);
  if (threadIdx.x == 0) {
    loss[t] = c;
    stats[2 * (size_t)t] = m;
    stats[2 * (size_t)t + 1] = l;
  }
}

template <class E>
__global__ __launch_bounds__(256) void distill_bwd_kernel(VocabDims d, const void* logits, const int* idx,
                                                          const float* teacher, const float* stats,
                                                          const float* g_loss, void* d_logits) {
  __shared__ float sh[4];
  __shared__ int lidx[256];
  __shared__ float lq[256];
  const int t = blockIdx.x, tid = threadIdx.x;
  const E* row = static_cast<const E*>(logits) + (size_t)t * d.ld;
  E* out = static_cast<E*>(d_logits) + (size_t)t * d.ldg;
  int ix;
  float qj, logq;
  bool any;
  teacher_row(d, t, idx, teacher, sh, ix, qj, logq, any);
  lidx[tid] = ix;
  lq[tid] = qj;
  __syncthreads();
  const float m = stats[2 * (size_t)t], l = stats[2 * (size_t)t + 1];
  const float g = g_loss[t];
  const bool bad = g != 0.0f && qj != qj;
  const bool none = g == 0.0f || bad || !any || l == -INFINITY;
  for (int i = tid; i < d.V; i += 256) {
    float v = bad ? NAN : 0.0f;
    if (!none) {
      const float p = __expf((to_f32<E>(row[i]) - m) * d.invtau - l);
      float qi = 0.0f;
      for (int j = 0; j < d.k; ++j) qi += lidx[j] == i ? lq[j] : 0.0f;
      v = g * (p - qi) * d.invtau;
    }
    if (d.accumulate) v += to_f32<E>(out[i]);
    out[i] = from_f32<E>(v);
  }
}

}  // namespace

size_t vocab_ws_bytes(const VocabDims&) { return 0; }

hipError_t launch_token_logprobs(const VocabDims& d, const LogprobPtrs& q, char*, hipStream_t st) {
  ProfScope prof(st, "vocab.logprobs");
  auto* f = d.f32 ? logprobs_kernel<float> : logprobs_kernel<uint16_t>;
  hipLaunchKernelGGL(f, dim3(d.T), dim3(256), 0, st, d, q);
  return hipGetLastError();
}

hipError_t launch_token_logprobs_bwd(const VocabDims& d, const LogprobGradPtrs& q, hipStream_t st) {
  ProfScope prof(st, "vocab.logprobs_bwd");
  auto* f = d.f32 ? logprobs_bwd_kernel<float> : logprobs_bwd_kernel<uint16_t>;
  hipLaunchKernelGGL(f, dim3(d.T), dim3(256), 0, st, d, q);
  return hipGetLastError();
}

hipError_t launch_distill(const VocabDims& d, const void* logits, const int* idx, const float* teacher, float* loss,
                          float* stats, char*, hipStream_t st) {
  ProfScope prof(st, "vocab.distill");
  auto* f = d.f32 ? distill_kernel<float> : distill_kernel<uint16_t>;
  hipLaunchKernelGGL(f, dim3(d.T), dim3(256), 0, st, d, logits, idx, teacher, loss, stats);
  return hipGetLastError();
}

hipError_t launch_distill_bwd(const VocabDims& d, const void* logits, const int* idx, const float* teacher,
                              const float* stats, const float* g_loss, void* d_logits, hipStream_t st) {
  ProfScope prof(st, "vocab.distill_bwd");
  auto* f = d.f32 ? distill_bwd_kernel<float> : distill_bwd_kernel<uint16_t>;
  hipLaunchKernelGGL(f, dim3(d.T), dim3(256), 0, st, d, logits, idx, teacher, stats, g_loss, d_logits);
  return hipGetLastError();
}

}  // namespace oft
