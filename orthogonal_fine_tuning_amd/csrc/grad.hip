// Global norm of many gradient tensors, and their clipping (oft_grad_sumsq /
// oft_grad_clip in oft.h).
//
//   sumsq = sum over all tensors of g^2,  norm = sqrt(sumsq),
//   coef = min(1, max_norm / (norm + 1e-6)),  out = coef g
// One read for the sum, one read and one write for the clipping: bound by
// those bytes.  The tensors' addresses travel in the kernel's arguments, up to
// 100 to a launch (or, for the host's sake, 12), so that nothing has to be
// copied to the GPU and a captured call replays.  Squares are added in fp64
// (two instructions an element, far below what the reads take): no finite
// gradient overflows, and the order of the chunks does not show in fp32.
#include "oft_device.h"
#include "oft_grad.h"
#include "oft_prof.h"

#include <type_traits>

namespace oft {
namespace {

constexpr float EPS = 1e-6f;
// Gradients of more bytes than this in all are streamed past the caches (norm
// and clipping into other tensors in us, streamed and not: 64 MB 38 and 42
// from memory, 35 and 35 from the caches, 120 MB 67, 78 and 64, 62, 512 MB 269
// and 308; 16 MB 13.5 and 12.6 from memory).  Where the two differ, gradients are
// taken to come from memory: most were written layers ago.
constexpr int64_t STREAM_BYTES = 64LL << 20;

struct Item {
  const void* g;
  void* out;
  int64_t n;
};
template <int N>
struct Items {
  static constexpr int MOST = N, WAVES = (N + 63) / 64;
  int first[64 * WAVES];  // chunk of the launch at which each tensor starts; INT_MAX past the last
  int count, chunks, chunk, pad;  // chunk: elements of one
  Item at[N];
};

// 16 bytes from an address that only its 4-byte alignment is known of
typedef uint32_t u32x4 __attribute__((ext_vector_type(4), aligned(4)));
template <bool STREAM>
__device__ __forceinline__ u32x4 load16(const u32x4* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(p);
  else return *p;
}
template <bool STREAM>
__device__ __forceinline__ void store16(u32x4* p, const u32x4& v) {
  if constexpr (STREAM) __builtin_nontemporal_store(v, p);
  else *p = v;
}

// The tensor of a chunk: the arguments lie in host memory, far away, so all
// the tensors' starts are looked at at once instead of by halves (585 MB in 48
// tensors: 141 us for the sum by halves).
template <int N>
__device__ __forceinline__ int item_of(const Items<N>& s, int chunk) {
  const int lane = threadIdx.x & 63;
  int before = 0;
#pragma unroll
  for (int i = 0; i < Items<N>::WAVES; ++i) before += __popcll(__ballot(s.first[64 * i + lane] <= chunk));
  return __builtin_amdgcn_readfirstlane(before - 1);
}

template <bool F32>
__device__ __forceinline__ float value(const void* p, int64_t i) {
  if constexpr (F32) return static_cast<const float*>(p)[i];
  else return bf16_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// elements in front of the first 4-byte aligned one (bf16 tensors may start
// between two)
template <bool F32>
__device__ __forceinline__ int odd_start(const void* p) {
  return F32 ? 0 : (int)((reinterpret_cast<uintptr_t>(p) >> 1) & 1);
}

// Elements [lo, hi) of g, by the 256 threads of a workgroup.
template <bool F32, bool STREAM>
__device__ __forceinline__ double sum_range(const void* g, int64_t lo, int64_t hi) {
  constexpr int E = F32 ? 4 : 8, U = 4;
  const int tid = threadIdx.x;
  const int64_t a = lo + odd_start<F32>(g);  // (lo is a multiple of 8)
  double s[2] = {0.0, 0.0};
  const int64_t vecs = hi > a ? (hi - a) / E : 0;
  const char* base = static_cast<const char*>(g) + a * (F32 ? 4 : 2);
  auto add = [&](const u32x4& v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (F32) {
        const double x = (double)__builtin_bit_cast(float, (uint32_t)v[k]);
        s[k & 1] = __builtin_fma(x, x, s[k & 1]);
      } else {
        // (the square of a bf16 is exact in fp32, short of its range)
        const double x = (double)__builtin_bit_cast(float, (uint32_t)v[k] << 16);
        const double y = (double)__builtin_bit_cast(float, (uint32_t)v[k] & 0xFFFF0000u);
        s[0] = __builtin_fma(x, x, s[0]);
        s[1] = __builtin_fma(y, y, s[1]);
      }
    }
  };
  int64_t i = tid;
  for (; i + (U - 1) * 256 < vecs; i += U * 256) {
    u32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = load16<STREAM>(reinterpret_cast<const u32x4*>(base) + i + u * 256);
#pragma unroll
    for (int u = 0; u < U; ++u) add(v[u]);
  }
  for (; i < vecs; i += 256) add(reinterpret_cast<const u32x4*>(base)[i]);
  // the element in front and those behind the vectors
  if (tid == 0 && a > lo && lo < hi) {
    const double x = (double)value<F32>(g, lo);
    s[0] = __builtin_fma(x, x, s[0]);
  }
  const int64_t t = a + vecs * E + tid;
  if (tid < E && t < hi) {
    const double x = (double)value<F32>(g, t);
    s[1] = __builtin_fma(x, x, s[1]);
  }
  return s[0] + s[1];
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// sum over the workgroup, in thread 0
template <int THREADS>
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double w[THREADS / 64];
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
#pragma unroll
    for (int i = 0; i < THREADS / 64; ++i) s += w[i];
  return s;
}

template <bool F32, bool STREAM, int N>
__global__ __launch_bounds__(256) void sumsq_kernel(Items<N> s, double* __restrict__ part) {
  const int i = item_of(s, blockIdx.x);
  const Item& t = s.at[i];
  const int64_t lo = (int64_t)((int)blockIdx.x - s.first[i]) * s.chunk;
  const double v = block_sum<256>(sum_range<F32, STREAM>(t.g, lo, min(t.n, lo + s.chunk)));
  if (threadIdx.x == 0) part[blockIdx.x] = v;
}

__global__ __launch_bounds__(1024) void sumsq_join_kernel(const double* __restrict__ part, int count,
                                                          double* __restrict__ sumsq) {
  double s = 0.0;
  for (int i = threadIdx.x; i < count; i += 1024) s += part[i];
  s = block_sum<1024>(s);
  if (threadIdx.x == 0) *sumsq = s;
}

// few elements in all: one workgroup, one launch
template <bool F32>
__global__ __launch_bounds__(256) void sumsq_few_kernel(Items<12> s, double* __restrict__ sumsq) {
  double v = 0.0;
  for (int i = 0; i < s.count; ++i) v += sum_range<F32, false>(s.at[i].g, 0, s.at[i].n);
  v = block_sum<256>(v);
  if (threadIdx.x == 0) *sumsq = v;
}

__device__ __forceinline__ float coefficient(const double* sumsq, float max_norm, float& norm) {
  norm = (float)sqrt(*sumsq);
  const float c = max_norm / (norm + EPS);
  if (norm == __builtin_inff()) return 0.0f;  // (also beside an infinite limit)
  return c > 1.0f ? 1.0f : c;                 // (NaN stays)
}

// out = c g over [lo, hi)
template <bool F32, bool STREAM>
__device__ __forceinline__ void scale_range(const void* g, void* out, int64_t lo, int64_t hi, float c) {
  constexpr int E = F32 ? 4 : 8, U = 4;
  const int tid = threadIdx.x;
  auto one = [&](int64_t i) {
    const float x = c * value<F32>(g, i);
    if constexpr (F32) static_cast<float*>(out)[i] = x;
    else static_cast<uint16_t*>(out)[i] = __builtin_bit_cast(uint16_t, (__bf16)x);
  };
  if (odd_start<F32>(g) != odd_start<F32>(out)) {  // no common 4-byte alignment
    for (int64_t i = lo + tid; i < hi; i += 256) one(i);
    return;
  }
  const int64_t a = lo + odd_start<F32>(g);
  const int64_t vecs = hi > a ? (hi - a) / E : 0;
  const u32x4* in = reinterpret_cast<const u32x4*>(static_cast<const char*>(g) + a * (F32 ? 4 : 2));
  u32x4* o = reinterpret_cast<u32x4*>(static_cast<char*>(out) + a * (F32 ? 4 : 2));
  auto scaled = [&](const u32x4& v) {
    u32x4 r;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (F32)
        r[k] = __builtin_bit_cast(uint32_t, c * __builtin_bit_cast(float, (uint32_t)v[k]));
      else
        r[k] = pack_bf16x2(c * __builtin_bit_cast(float, (uint32_t)v[k] << 16),
                           c * __builtin_bit_cast(float, (uint32_t)v[k] & 0xFFFF0000u));
    }
    return r;
  };
  int64_t i = tid;
  for (; i + (U - 1) * 256 < vecs; i += U * 256) {
    u32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = load16<STREAM>(in + i + u * 256);
#pragma unroll
    for (int u = 0; u < U; ++u) store16<STREAM>(o + i + u * 256, scaled(v[u]));
  }
  for (; i < vecs; i += 256) o[i] = scaled(in[i]);
  if (tid == 0 && a > lo && lo < hi) one(lo);
  const int64_t t = a + vecs * E + tid;
  if (tid < E && t < hi) one(t);
}

template <bool F32, bool STREAM, int N>
__global__ __launch_bounds__(256) void clip_kernel(Items<N> s, const double* __restrict__ sumsq, float max_norm,
                                                   float* __restrict__ stats) {
  float norm;
  const float c = coefficient(sumsq, max_norm, norm);
  if (blockIdx.x == 0 && threadIdx.x == 0 && stats != nullptr) {
    stats[0] = norm;
    stats[1] = c;
  }
  if (s.count == 0) return;
  const int i = item_of(s, blockIdx.x);
  const Item& t = s.at[i];
  if (c == 1.0f && t.out == t.g) return;
  const int64_t lo = (int64_t)((int)blockIdx.x - s.first[i]) * s.chunk;
  scale_range<F32, STREAM>(t.g, t.out, lo, min(t.n, lo + s.chunk), c);
}

// Elements a workgroup takes: 16384, fewer where that leaves the chip idle.
int chunk_of(int m, const int64_t* numel) {
  int64_t total = 0;
  for (int i = 0; i < m; ++i) total += numel[i];
  int chunk = 16384;
  while (chunk > 1024 && total / chunk < 1024) chunk /= 2;
  return chunk;
}
constexpr int64_t FEW = 16384;

// f(items) for each launch's worth of tensors that are not empty, and the
// chunks before it
template <int N, class F>
void launches_of(const GradList& l, void* const* out, F f) {
  Items<N> s;
  s.chunk = chunk_of(l.m, l.numel);
  int before = 0;
  for (int i = 0; i < l.m;) {
    s.count = s.chunks = 0;
    for (; i < l.m && s.count < N; ++i) {
      if (l.numel[i] == 0) continue;
      s.first[s.count] = s.chunks;
      s.at[s.count++] = Item{l.grads[i], out != nullptr ? out[i] : nullptr, l.numel[i]};
      s.chunks += (int)((l.numel[i] + s.chunk - 1) / s.chunk);
    }
    for (int k = s.count; k < 64 * Items<N>::WAVES; ++k) s.first[k] = 0x7FFFFFFF;
    if (s.count > 0) f(s, before);
    before += s.chunks;
  }
}

template <class F>
void launches(const GradList& l, void* const* out, F f) {
  if (l.m <= 12) launches_of<12>(l, out, f);
  else launches_of<100>(l, out, f);
}

int64_t chunks_of(int m, const int64_t* numel) {
  const int chunk = chunk_of(m, numel);
  int64_t c = 0;
  for (int i = 0; i < m; ++i) c += (numel[i] + chunk - 1) / chunk;
  return c;
}

int64_t total_of(const GradList& l) {
  int64_t total = 0;
  for (int i = 0; i < l.m; ++i) total += l.numel[i];
  return total;
}
bool few(const GradList& l) { return l.m <= 12 && total_of(l) <= FEW; }
bool streamed(const GradList& l) { return total_of(l) * (l.f32 ? 4 : 2) > STREAM_BYTES; }

template <class F>
void choose(bool a, bool b, F f) {
  if (a) b ? f(std::true_type{}, std::true_type{}) : f(std::true_type{}, std::false_type{});
  else b ? f(std::false_type{}, std::true_type{}) : f(std::false_type{}, std::false_type{});
}

}  // namespace

size_t grad_ws_bytes(int m, const int64_t* numel) { return 8 * (size_t)chunks_of(m, numel); }

hipError_t launch_grad_sumsq(const GradList& l, double* sumsq, char* ws, hipStream_t st) {
  ProfScope prof(st, "grad.sumsq");
  if (few(l)) {
    bool any = false;
    launches_of<12>(l, nullptr, [&](const Items<12>& s, int) {
      any = true;
      if (l.f32) hipLaunchKernelGGL(sumsq_few_kernel<true>, dim3(1), dim3(256), 0, st, s, sumsq);
      else hipLaunchKernelGGL(sumsq_few_kernel<false>, dim3(1), dim3(256), 0, st, s, sumsq);
    });
    if (any) return hipGetLastError();
  }
  double* part = reinterpret_cast<double*>(ws);
  launches(l, nullptr, [&](const auto& s, int before) {
    constexpr int N = std::remove_reference_t<decltype(s)>::MOST;
    choose(l.f32, streamed(l), [&](auto f32, auto stream) {
      hipLaunchKernelGGL((sumsq_kernel<decltype(f32)::value, decltype(stream)::value, N>), dim3(s.chunks), dim3(256), 0, st,
                         s, part + before);
    });
  });
  hipLaunchKernelGGL(sumsq_join_kernel, dim3(1), dim3(1024), 0, st, part, (int)chunks_of(l.m, l.numel), sumsq);
  return hipGetLastError();
}

hipError_t launch_grad_clip(const GradList& l, const double* sumsq, float max_norm, void* const* out, float* stats,
                            hipStream_t st) {
  ProfScope prof(st, "grad.clip");
  bool first = true;
  auto run = [&](const auto& s, int) {
    constexpr int N = std::remove_reference_t<decltype(s)>::MOST;
    float* to = first ? stats : nullptr;
    first = false;
    const dim3 grid(s.chunks > 0 ? s.chunks : 1);
    choose(l.f32, streamed(l), [&](auto f32, auto stream) {
      hipLaunchKernelGGL((clip_kernel<decltype(f32)::value, decltype(stream)::value, N>), grid, dim3(256), 0, st, s, sumsq,
                         max_norm, to);
    });
  };
  launches(l, out, run);
  if (first) {  // nothing to scale: the norm and coefficient alone
    Items<12> s;
    s.count = s.chunks = 0;
    s.chunk = 1;
    run(s, 0);
  }
  return hipGetLastError();
}

}  // namespace oft
