// Losses on vocabulary logits (include/oft.h): log-probabilities of given
// tokens with entropy and top alternatives, distillation from a teacher's
// top logits, and their gradients.
//
// With x a row, m its maximum and c = log2(e) / tau:
//   e_i = 2^(c (x_i - m)), s = sum e_i, w = sum e_i (x_i - m),
//   l = ln s, log p_i = (x_i - m) / tau - l, H = l - w / (tau s).
// A sum over part of a row is the triple (m, s, w) with its own m; moving it
// to a larger maximum M multiplies s by f = 2^(c (m - M)) and turns w into
// f (w + s (m - M)).
//
// Forward: vocab_stats_kernel reads every logit once (the operator is bound
// by that read) and leaves one triple per slice of a row and, for the top
// alternatives, the maximum of every 64 consecutive columns;
// logprobs_finish_kernel / distill_finish_kernel join a row's slices.  The k
// largest logits all lie in the k best of the 64-column blocks (order: larger
// maximum, then lower block): a block outside has k blocks before it, each
// with an element that beats all of its own.  So only k blocks of a row are
// read again.
//
// Backward: one read and one write per logit with (m, l) from the forward.
//
// Rows start anywhere (16-byte loads at element alignment, which gfx950
// allows); only a row's last, partial vector is read by elements, so nothing
// outside a row is touched.
#include <math.h>

#include "oft_device.h"
#include "oft_launch.h"
#include "oft_prof.h"
#include "oft_vocab.h"

namespace oft {
namespace {

constexpr float LOG2E = 1.44269504088896340736f;
constexpr float LN2 = 0.69314718055994530942f;
// clamp of z and log p where they are multiplied by p: p is 0 in fp32 far
// above it, and 0 times it is 0 (0 times -inf would be NaN)
constexpr float LOWEST = -1000.0f;
// the same for x - m where it meets a weight that is 0 from far above it on
// (tau <= 2^20), so that a sum of masks at the type's lowest value stays finite
constexpr float FAR = -1.0e30f;
constexpr int BLOCK = 64;  // columns per stored maximum

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_row __attribute__((aligned(2), may_alias));  // 16 bytes of a row

// a logit type: E, its 16-byte vectors of VE elements
struct Bf16 {
  typedef uint16_t E;
  static constexpr int VE = 8;
  static __device__ __forceinline__ float get(E v) { return bf16_to_f32(v); }
  static __device__ __forceinline__ E put(float v) { return (E)(pack_bf16x2(v, 0.0f) & 0xFFFFu); }
  static __device__ __forceinline__ void unpack(const u32x4& v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __builtin_bit_cast(float, v[i] << 16);
      f[2 * i + 1] = __builtin_bit_cast(float, v[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float* f) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    return v;
  }
};
struct F32 {
  typedef float E;
  static constexpr int VE = 4;
  static __device__ __forceinline__ float get(E v) { return v; }
  static __device__ __forceinline__ E put(float v) { return v; }
  static __device__ __forceinline__ void unpack(const u32x4& v, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = v[i];  // (a bit_cast of the element itself takes element 0)
      f[i] = __builtin_bit_cast(float, w);
    }
  }
  static __device__ __forceinline__ u32x4 pack(const float* f) {
    u32x4 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __builtin_bit_cast(uint32_t, f[i]);
    return v;
  }
};

__device__ __forceinline__ float exp2_hw(float v) { return __builtin_amdgcn_exp2f(v); }

template <class E>
__device__ __forceinline__ u32x4 load16(const E* p) {
  return *reinterpret_cast<const u32x4_row*>(p);
}
template <class E>
__device__ __forceinline__ void store16(E* p, const u32x4& v) {
  *reinterpret_cast<u32x4_row*>(p) = v;
}

// lane-wise maximum with another lane of the same 16 (DPP)
template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
  const int o = __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, v), __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, false);
  return fmaxf(v, __builtin_bit_cast(float, o));
}

// ------------------------------------------------------------------ triples
struct Triple {
  float m, s, w;
};

// the triple of both sets; an empty set has s = 0
__device__ __forceinline__ Triple join(const Triple& a, const Triple& b, float c) {
  if (b.s == 0.0f) return a;
  if (a.s == 0.0f) return b;
  const float M = fmaxf(a.m, b.m), da = a.m - M, db = b.m - M;
  const float fa = exp2_hw(c * da), fb = exp2_hw(c * db);
  return Triple{M, fmaf(a.s, fa, b.s * fb),
                fa * fmaf(a.s, fmaxf(da, FAR), a.w) + fb * fmaf(b.s, fmaxf(db, FAR), b.w)};
}

__device__ __forceinline__ Triple wave_join(Triple a, float c) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    const Triple b{__shfl_xor(a.m, off), __shfl_xor(a.s, off), __shfl_xor(a.w, off)};
    // the lower lane's set comes first on both sides, so both get the same bits
    a = (threadIdx.x & off) ? join(b, a, c) : join(a, b, c);
  }
  return a;
}

// ------------------------------------------------------------- forward pass
constexpr int FU = 4;  // vectors per thread and step

template <class Ty>
constexpr int fwd_tile() {
  return 256 * FU * Ty::VE;
}

// one step: FU vectors per thread, x[u VE + j] is column base + (u 256 + tid) VE + j
template <class Ty, bool ENT, bool TOP>
__device__ __forceinline__ void fwd_step(const float (&x)[FU * Ty::VE], int base, int V, float c, Triple& a,
                                         typename Ty::E* blocks) {
  constexpr int VE = Ty::VE, N = FU * VE;
  float vm[FU];
#pragma unroll
  for (int u = 0; u < FU; ++u) {
    vm[u] = x[u * VE];
#pragma unroll
    for (int j = 1; j < VE; ++j) vm[u] = fmaxf(vm[u], x[u * VE + j]);
  }
  float bm = vm[0];
#pragma unroll
  for (int u = 1; u < FU; ++u) bm = fmaxf(bm, vm[u]);
  // larger maximum: move the sums to it (from -inf: they are 0)
  const float M = fmaxf(a.m, bm);
  const float d0 = a.s == 0.0f ? 0.0f : a.m - M;
  const float f = exp2_hw(c * d0);
  a.w = f * fmaf(a.s, fmaxf(d0, FAR), a.w);
  a.s *= f;
  a.m = M;
  const float ref = M == -INFINITY ? 0.0f : M;
  float s[2] = {0.0f, 0.0f}, w[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float d = x[i] - ref;
    const float e = exp2_hw(c * d);
    s[i & 1] += e;
    if constexpr (ENT) w[i & 1] = fmaf(e, fmaxf(d, FAR), w[i & 1]);
  }
  a.s += s[0] + s[1];
  a.w += w[0] + w[1];
  if constexpr (TOP) {
    // 64 columns are 64 / VE neighbouring lanes of one vector
    constexpr int G = BLOCK / VE;
    const int lane = threadIdx.x & 63;
    float mine = -INFINITY;
#pragma unroll
    for (int u = 0; u < FU; ++u) {
      float v = dpp_max<0xB1>(vm[u]);   // lanes of a pair
      v = dpp_max<0x4E>(v);             // of a quad
      v = dpp_max<0x141>(v);            // of eight
      if constexpr (G == 16) v = dpp_max<0x140>(v);
      mine = (lane % G) == u ? v : mine;
    }
    // lane u of a group stores the block of vector u
    if (lane % G < FU) {
      const int b = (base + ((lane % G) * 256 + threadIdx.x - lane % G) * VE) / BLOCK;
      if (b * BLOCK < V) blocks[b] = Ty::put(mine);
    }
  }
}

// part[t S + sl]: the triple of columns [sl slice, (sl + 1) slice) of row t;
// blocks: the maxima of the row's 64-column blocks, nb per row
template <class Ty, bool ENT, bool TOP>
__global__ __launch_bounds__(256) void vocab_stats_kernel(const typename Ty::E* __restrict__ logits, long ld, int V,
                                                          int S, int slice, float c, float4* __restrict__ part,
                                                          typename Ty::E* __restrict__ blocks, int nb) {
  typedef typename Ty::E E;
  constexpr int VE = Ty::VE, TILE = fwd_tile<Ty>();
  __shared__ float sh[4][3];
  const int t = blockIdx.x / S, sl = blockIdx.x % S, tid = threadIdx.x;
  const E* row = logits + (size_t)t * ld;
  E* brow = TOP ? blocks + (size_t)t * nb : nullptr;
  const int lo = sl * slice, hi = min(V, lo + slice);
  Triple a{-INFINITY, 0.0f, 0.0f};
  float x[FU * VE];
  int base = lo;
  for (; base + TILE <= hi; base += TILE) {
    u32x4 v[FU];
#pragma unroll
    for (int u = 0; u < FU; ++u) v[u] = load16(row + base + (u * 256 + tid) * VE);
#pragma unroll
    for (int u = 0; u < FU; ++u) Ty::unpack(v[u], x + u * VE);
    fwd_step<Ty, ENT, TOP>(x, base, V, c, a, brow);
  }
  if (base < hi) {
#pragma unroll
    for (int u = 0; u < FU; ++u) {
      const int i0 = base + (u * 256 + tid) * VE;
      if (i0 + VE <= hi) {
        Ty::unpack(load16(row + i0), x + u * VE);
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j) x[u * VE + j] = i0 + j < hi ? Ty::get(row[i0 + j]) : -INFINITY;
      }
    }
    fwd_step<Ty, ENT, TOP>(x, base, V, c, a, brow);
  }
  a = wave_join(a, c);
  if ((tid & 63) == 0) {
    sh[tid >> 6][0] = a.m;
    sh[tid >> 6][1] = a.s;
    sh[tid >> 6][2] = a.w;
  }
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < 4; ++i) a = join(a, Triple{sh[i][0], sh[i][1], sh[i][2]}, c);
    part[blockIdx.x] = make_float4(a.m, a.s, a.w, 0.0f);
  }
}

// a row's triple from its slices, in every lane of the wave
__device__ __forceinline__ Triple row_triple(const float4* part, int S, float c) {
  Triple a{-INFINITY, 0.0f, 0.0f};
  for (int i = threadIdx.x & 63; i < S; i += 64) {
    const float4 p = part[i];
    a = join(a, Triple{p.x, p.y, p.z}, c);
  }
  return wave_join(a, c);
}

// ---------------------------------------------------------- top alternatives
// A wave's selection of the k best of a stream of (value, id), ids ascending:
// candidates wait in LDS in order of id; when the list is full it is cut to
// its k best, whose last value is then what a later candidate must exceed.
constexpr int QCAP = 512, MAXTOP = 128;

__device__ __forceinline__ uint32_t ordered(float v) {  // unsigned order of values
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.0f);  // -0 as +0
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __builtin_bit_cast(float, (o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}

__device__ __forceinline__ int below(unsigned long long mask) {  // set bits of lower lanes
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// k-th largest of the N lane values (in `ordered` form)
template <int N>
__device__ __forceinline__ uint32_t kth(const uint32_t (&o)[N], int k) {
  uint32_t r = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t tryv = r | (1u << bit);
    int n = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) n += __popcll(__ballot(o[j] >= tryv));
    if (n >= k) r = tryv;
  }
  return r;
}

struct Select {
  float* val;  // [QCAP] in LDS
  int* id;     // [QCAP]
  int k, n;
  float floor;  // a candidate must reach it, or exceed it once `strict`
  bool strict;

  __device__ __forceinline__ Select(float* v, int* i, int kk, float f) : val(v), id(i), k(kk), n(0), floor(f), strict(false) {}

  __device__ __forceinline__ void feed(float v, int i, bool ok) {
    const bool take = ok && (strict ? v > floor : v >= floor);
    const unsigned long long mask = __ballot(take);
    if (mask == 0) return;
    if (take) {
      const int at = n + below(mask);
      val[at] = v;
      id[at] = i;
    }
    n += __popcll(mask);
    if (n > QCAP - 64) cut();
  }

  // keep the k best, in order of id
  __device__ void cut() {
    __syncthreads();
    if (n <= k) return;
    constexpr int N = QCAP / 64;
    const int lane = threadIdx.x & 63;
    uint32_t o[N];
    int ids[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const bool in = j * 64 + lane < n;
      o[j] = in ? ordered(val[j * 64 + lane]) : 0u;
      ids[j] = in ? id[j * 64 + lane] : 0;
    }
    const uint32_t last = kth<N>(o, k);
    int above = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) above += __popcll(__ballot(o[j] > last));
    int ties = k - above, m = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const unsigned long long eq = __ballot(o[j] == last && j * 64 + lane < n);
      const bool keep = o[j] > last || (o[j] == last && j * 64 + lane < n && below(eq) < ties);
      const unsigned long long mask = __ballot(keep);
      if (keep) {
        val[m + below(mask)] = unordered(o[j]);
        id[m + below(mask)] = ids[j];
      }
      m += __popcll(mask);
      ties -= min(ties, (int)__popcll(eq));
    }
    n = m;
    floor = unordered(last);
    strict = true;
    __syncthreads();
  }
};

template <class Ty>
__device__ __forceinline__ float rank_value(typename Ty::E v) {  // NaN ranks as -inf
  const float f = Ty::get(v);
  return f != f ? -INFINITY : f;
}

struct FinishArgs {
  int V, k, S, nb;
  long ld;
  float c, invtau;
};

// one wave per row
template <class Ty, bool TOP>
__global__ __launch_bounds__(64) void logprobs_finish_kernel(FinishArgs f, LogprobPtrs q,
                                                             const float4* __restrict__ part,
                                                             const typename Ty::E* __restrict__ blocks) {
  typedef typename Ty::E E;
  const int t = blockIdx.x, lane = threadIdx.x;
  const E* row = static_cast<const E*>(q.logits) + (size_t)t * f.ld;
  const Triple a = row_triple(part + (size_t)t * f.S, f.S, f.c);
  const bool empty = a.s == 0.0f;
  const float l = __logf(a.s);  // ln 0 = -inf for an empty row
  if (lane == 0) {
    *reinterpret_cast<float2*>(q.stats + 2 * (size_t)t) = make_float2(a.m, l);
    if (q.entropy) q.entropy[t] = empty ? 0.0f : l - a.w * f.invtau / a.s;
    if (q.logp) {
      const int lab = q.labels[t];
      float lp = lab == -1 ? 0.0f : NAN;
      if (lab >= 0 && lab < f.V) lp = empty ? -INFINITY : (Ty::get(row[lab]) - a.m) * f.invtau - l;
      q.logp[t] = lp;
    }
  }
  if constexpr (TOP) {
    __shared__ float val[2][QCAP];
    __shared__ int id[2][QCAP];
    const E* brow = blocks + (size_t)t * f.nb;
    // a value that at least k blocks reach: the k-th best of 128 interleaved
    // groups of blocks
    float best[2] = {-INFINITY, -INFINITY};
    for (int b = lane; b < f.nb; b += 128) {
      best[0] = fmaxf(best[0], Ty::get(brow[b]));
      if (b + 64 < f.nb) best[1] = fmaxf(best[1], Ty::get(brow[b + 64]));
    }
    const uint32_t o[2] = {ordered(best[0]), ordered(best[1])};
    Select sel(val[0], id[0], f.k, unordered(kth<2>(o, f.k)));
    for (int b = 0; b < f.nb; b += 64) {
      const bool in = b + lane < f.nb;
      sel.feed(in ? rank_value<Ty>(brow[b + lane]) : 0.0f, b + lane, in);
    }
    sel.cut();
    __syncthreads();
    // their elements: at least k reach the least of k maxima
    const int nsel = sel.n;
    float lowest = INFINITY;
    for (int i = lane; i < nsel; i += 64) lowest = fminf(lowest, val[0][i]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) lowest = fminf(lowest, __shfl_xor(lowest, off));
    Select el(val[1], id[1], f.k, nsel < f.k ? -INFINITY : lowest);
    for (int i = 0; i < nsel; i += 8) {
      float v[8];
      int col[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        col[j] = i + j < nsel ? id[0][i + j] * BLOCK + lane : f.V;
        v[j] = col[j] < f.V ? rank_value<Ty>(row[col[j]]) : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) el.feed(v[j], col[j], col[j] < f.V);
    }
    el.cut();
    __syncthreads();
    // best first: an entry's place is the number of entries before it
#pragma unroll
    for (int h = 0; h < MAXTOP / 64; ++h) {
      const int i = h * 64 + lane;
      if (i < f.k) {
        const float v = val[1][i];
        int place = 0;
        for (int j = 0; j < f.k; ++j) {
          const float u = val[1][j];
          place += (u > v || (u == v && j < i)) ? 1 : 0;
        }
        const size_t at = (size_t)t * f.k + place;
        q.top_idx[at] = id[1][i];
        q.top_logp[at] = l != l ? NAN : empty ? -INFINITY : (v - a.m) * f.invtau - l;
      }
    }
  }
}

// ------------------------------------------------------------------ teacher
// A row's teacher list over one wave: entry lane + 64 i in register i.
// ix -1: an entry without weight.  bad: an entry is out of range, NaN or
// +inf; any: some entry has weight.
constexpr int TI = 4;
struct Teacher {
  int ix[TI];
  float q[TI], logq[TI];
  bool bad, any;

  __device__ __forceinline__ Teacher(const int* idx, const float* val, int k, int V, float invtau) {
    const int lane = threadIdx.x & 63;
    float v[TI], mx = -INFINITY;
    bool b = false;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      ix[i] = -1;
      v[i] = -INFINITY;
      if (lane + 64 * i < k) {
        ix[i] = idx[lane + 64 * i];
        if (ix[i] != -1) v[i] = val[lane + 64 * i];
        b |= ix[i] < -1 || ix[i] >= V || v[i] != v[i] || v[i] == INFINITY;
      }
      mx = fmaxf(mx, v[i]);
    }
    bad = __ballot(b) != 0;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) mx = fmaxf(mx, __shfl_xor(mx, off));
    any = mx != -INFINITY;
    float s = 0.0f, e[TI];
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      logq[i] = any ? (v[i] - mx) * invtau : -INFINITY;
      e[i] = exp2_hw(logq[i] * LOG2E);
      s += e[i];
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) s += __shfl_xor(s, off);
    const float ls = __logf(s);
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      q[i] = any ? e[i] / s : 0.0f;
      logq[i] -= ls;
      if (!(q[i] > 0.0f) || bad) ix[i] = -1;
    }
  }
};

// one wave per row
template <class Ty>
__global__ __launch_bounds__(64) void distill_finish_kernel(FinishArgs f, const typename Ty::E* __restrict__ logits,
                                                            const int* __restrict__ idx,
                                                            const float* __restrict__ teacher,
                                                            const float4* __restrict__ part, float* __restrict__ loss,
                                                            float* __restrict__ stats) {
  const int t = blockIdx.x;
  const typename Ty::E* row = logits + (size_t)t * f.ld;
  const Teacher te(idx + (size_t)t * f.k, teacher + (size_t)t * f.k, f.k, f.V, f.invtau);
  float x[TI];
#pragma unroll
  for (int i = 0; i < TI; ++i) x[i] = te.ix[i] >= 0 ? Ty::get(row[te.ix[i]]) : 0.0f;
  const Triple a = row_triple(part + (size_t)t * f.S, f.S, f.c);
  const float l = __logf(a.s);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < TI; ++i)
    if (te.ix[i] >= 0) {
      const float lp = a.s == 0.0f ? -INFINITY : (x[i] - a.m) * f.invtau - l;
      sum = fmaf(te.q[i], te.logq[i] - lp, sum);
    }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
  if (threadIdx.x == 0) {
    loss[t] = te.bad ? NAN : sum;
    *reinterpret_cast<float2*>(stats + 2 * (size_t)t) = make_float2(a.m, l);
  }
}

// ----------------------------------------------------------------- backward
// d_logits = p fma(max(log2 p, clamp), ga, gb) (+ gl / tau at the label) with
// log2 p = c (x - m) - l log2 e:
//   logprobs  ga = -g_H ln 2 / tau, gb = -(g_logp + g_H H) / tau
//   distill   ga = 0, gb = g / tau (the listed columns follow)
constexpr int BU = 4;  // vectors per thread and step

template <class Ty>
constexpr int bwd_tile() {
  return 256 * BU * Ty::VE;
}

struct RowGrad {
  float m, c, l2, ga, gb;
  __device__ __forceinline__ float log2p(float x) const { return fmaf(x - m, c, -l2); }
  __device__ __forceinline__ float operator()(float x) const {
    const float lp = log2p(x);
    return exp2_hw(lp) * fmaf(fmaxf(lp, LOWEST), ga, gb);
  }
};

enum { FILL_NONE = 0, FILL_ZERO = 1, FILL_NAN = 2 };

// columns [lo, hi) of a row: the gradient, or the same value everywhere
template <class Ty, bool ACC, class F>
__device__ __forceinline__ void bwd_columns(const typename Ty::E* row, typename Ty::E* out, int lo, int hi, int fill,
                                            F grad) {
  typedef typename Ty::E E;
  constexpr int VE = Ty::VE, TILE = bwd_tile<Ty>();
  const int tid = threadIdx.x;
  if (fill == FILL_ZERO && ACC) return;  // adds nothing
  if (fill != FILL_NONE) {
    const float v = fill == FILL_ZERO ? 0.0f : NAN;
    float f[VE];
#pragma unroll
    for (int j = 0; j < VE; ++j) f[j] = v;
    const u32x4 p = Ty::pack(f);
    for (int i0 = lo + tid * VE; i0 < hi; i0 += 256 * VE) {
      if (i0 + VE <= hi) {
        store16(out + i0, p);
      } else {
        for (int j = 0; i0 + j < hi; ++j) out[i0 + j] = Ty::put(v);
      }
    }
    return;
  }
  int base = lo;
  for (; base + TILE <= hi; base += TILE) {
    u32x4 v[BU], old[BU];
#pragma unroll
    for (int u = 0; u < BU; ++u) {
      v[u] = load16(row + base + (u * 256 + tid) * VE);
      if constexpr (ACC) old[u] = load16(out + base + (u * 256 + tid) * VE);
    }
#pragma unroll
    for (int u = 0; u < BU; ++u) {
      const int i0 = base + (u * 256 + tid) * VE;
      float x[VE], o[VE];
      Ty::unpack(v[u], x);
      if constexpr (ACC) Ty::unpack(old[u], o);
#pragma unroll
      for (int j = 0; j < VE; ++j) x[j] = grad(x[j], i0 + j) + (ACC ? o[j] : 0.0f);
      store16(out + i0, Ty::pack(x));
    }
  }
  for (int i0 = base + tid * VE; i0 < hi; i0 += 256 * VE) {
    float x[VE], o[VE];
    if (i0 + VE <= hi) {
      Ty::unpack(load16(row + i0), x);
      if constexpr (ACC) Ty::unpack(load16(out + i0), o);
#pragma unroll
      for (int j = 0; j < VE; ++j) x[j] = grad(x[j], i0 + j) + (ACC ? o[j] : 0.0f);
      store16(out + i0, Ty::pack(x));
    } else {
      for (int i = i0; i < hi; ++i) {
        const float v = grad(Ty::get(row[i]), i) + (ACC ? Ty::get(out[i]) : 0.0f);
        out[i] = Ty::put(v);
      }
    }
  }
}

struct BwdArgs {
  int V, k, S, slice;
  long ld, ldg;
  float c, invtau;
};

template <class Ty, bool ACC>
__global__ __launch_bounds__(256) void logprobs_bwd_kernel(BwdArgs b, LogprobGradPtrs q) {
  typedef typename Ty::E E;
  const int t = blockIdx.x / b.S, sl = blockIdx.x % b.S;
  const E* row = static_cast<const E*>(q.logits) + (size_t)t * b.ld;
  E* out = static_cast<E*>(q.d_logits) + (size_t)t * b.ldg;
  const int lo = sl * b.slice, hi = min(b.V, lo + b.slice);
  const float2 st = *reinterpret_cast<const float2*>(q.stats + 2 * (size_t)t);
  const int lab = q.labels ? q.labels[t] : -1;
  const float gl = lab == -1 ? 0.0f : q.g_logp[t];
  const float ge = q.g_entropy ? q.g_entropy[t] : 0.0f;
  const float H = ge != 0.0f ? q.entropy[t] : 0.0f;
  int fill = FILL_NONE;
  if (gl == 0.0f && ge == 0.0f) fill = FILL_ZERO;
  else if (lab < -1 || lab >= b.V) fill = FILL_NAN;
  else if (st.y == -INFINITY) fill = FILL_ZERO;
  const RowGrad g{st.x, b.c, st.y * LOG2E, -ge * LN2 * b.invtau, -fmaf(ge, H, gl) * b.invtau};
  const float at = gl * b.invtau;
  bwd_columns<Ty, ACC>(row, out, lo, hi, fill,
                       [&](float x, int i) { return g(x) + (i == lab ? at : 0.0f); });
}

template <class Ty, bool ACC>
__global__ __launch_bounds__(256) void distill_bwd_kernel(BwdArgs b, const typename Ty::E* logits,
                                                          const int* __restrict__ idx,
                                                          const float* __restrict__ teacher,
                                                          const float* __restrict__ stats,
                                                          const float* __restrict__ g_loss, typename Ty::E* d_logits) {
  typedef typename Ty::E E;
  __shared__ int lidx[64 * TI];
  __shared__ float lq[64 * TI];
  const int t = blockIdx.x / b.S, sl = blockIdx.x % b.S, tid = threadIdx.x;
  const E* row = logits + (size_t)t * b.ld;
  E* out = d_logits + (size_t)t * b.ldg;
  const int lo = sl * b.slice, hi = min(b.V, lo + b.slice);
  const float2 st = *reinterpret_cast<const float2*>(stats + 2 * (size_t)t);
  const float g = g_loss[t];
  // (each wave computes the list; all get the same)
  const Teacher te(idx + (size_t)t * b.k, teacher + (size_t)t * b.k, b.k, b.V, b.invtau);
  if (tid < 64) {
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      lidx[tid + 64 * i] = te.ix[i];
      lq[tid + 64 * i] = te.q[i];
    }
  }
  int fill = FILL_NONE;
  if (g == 0.0f) fill = FILL_ZERO;
  else if (te.bad) fill = FILL_NAN;
  else if (!te.any || st.y == -INFINITY) fill = FILL_ZERO;
  __syncthreads();
  const RowGrad r{st.x, b.c, st.y * LOG2E, 0.0f, g * b.invtau};
  // the listed columns of this slice, one per thread: p - sum of their q.
  // Read before anything is written (d_logits may be logits)
  const int mine = lidx[tid];
  const bool listed = fill == FILL_NONE && mine >= lo && mine < hi;
  float v = 0.0f;
  if (listed) {
    float q = 0.0f;
    for (int j = 0; j < b.k; ++j) q += lidx[j] == mine ? lq[j] : 0.0f;
    v = (exp2_hw(r.log2p(Ty::get(row[mine]))) - q) * r.gb;
    if constexpr (ACC) v += Ty::get(out[mine]);
  }
  __syncthreads();
  bwd_columns<Ty, ACC>(row, out, lo, hi, fill, [&](float x, int) { return exp2_hw(r.log2p(x)) * r.gb; });
  __syncthreads();  // the slice's own writes come before the listed columns'
  if (listed) out[mine] = Ty::put(v);
}

// --------------------------------------------------------------- host side
// Slices of a row: enough workgroups to fill the chip several times over, at
// least a tile each.
struct Split {
  int S, slice;
};
Split split(int T, int V, int tile) {
  const long tiles = ((long)V + tile - 1) / tile;
  const long want = (8192 + T - 1) / T;
  const long S = want < tiles ? want : tiles;
  const long per = (tiles + S - 1) / S;
  return Split{(int)((tiles + per - 1) / per), (int)(per * tile)};
}
Split fwd_split(const VocabDims& d) { return split(d.T, d.V, d.f32 ? fwd_tile<F32>() : fwd_tile<Bf16>()); }
Split bwd_split(const VocabDims& d) { return split(d.T, d.V, d.f32 ? bwd_tile<F32>() : bwd_tile<Bf16>()); }

int blocks_of(int V) { return (V + BLOCK - 1) / BLOCK; }
size_t part_bytes(const VocabDims& d) { return (size_t)d.T * fwd_split(d).S * sizeof(float4); }

FinishArgs finish_args(const VocabDims& d, int S) {
  return FinishArgs{d.V, d.k, S, blocks_of(d.V), d.ld, d.invtau * LOG2E, d.invtau};
}
BwdArgs bwd_args(const VocabDims& d) {
  const Split s = bwd_split(d);
  return BwdArgs{d.V, d.k, s.S, s.slice, d.ld, d.ldg, d.invtau * LOG2E, d.invtau};
}

template <class Ty, bool ENT, bool TOP>
void stats_launch(const VocabDims& d, const Split& s, const void* logits, char* ws, hipStream_t st) {
  typedef typename Ty::E E;
  hipLaunchKernelGGL((vocab_stats_kernel<Ty, ENT, TOP>), dim3((size_t)d.T * s.S), dim3(256), 0, st,
                     static_cast<const E*>(logits), d.ld, d.V, s.S, s.slice, d.invtau * LOG2E,
                     reinterpret_cast<float4*>(ws), reinterpret_cast<E*>(ws + part_bytes(d)), blocks_of(d.V));
}

template <class Ty>
void logprobs_launch(const VocabDims& d, const LogprobPtrs& q, char* ws, hipStream_t st) {
  const Split s = fwd_split(d);
  const float4* part = reinterpret_cast<const float4*>(ws);
  const typename Ty::E* blocks = reinterpret_cast<const typename Ty::E*>(ws + part_bytes(d));
  const FinishArgs f = finish_args(d, s.S);
  if (d.k > 0) {
    if (q.entropy) stats_launch<Ty, true, true>(d, s, q.logits, ws, st);
    else stats_launch<Ty, false, true>(d, s, q.logits, ws, st);
    hipLaunchKernelGGL((logprobs_finish_kernel<Ty, true>), dim3(d.T), dim3(64), 0, st, f, q, part, blocks);
  } else {
    if (q.entropy) stats_launch<Ty, true, false>(d, s, q.logits, ws, st);
    else stats_launch<Ty, false, false>(d, s, q.logits, ws, st);
    hipLaunchKernelGGL((logprobs_finish_kernel<Ty, false>), dim3(d.T), dim3(64), 0, st, f, q, part, blocks);
  }
}

template <class Ty>
void distill_launch(const VocabDims& d, const void* logits, const int* idx, const float* teacher, float* loss,
                    float* stats, char* ws, hipStream_t st) {
  const Split s = fwd_split(d);
  stats_launch<Ty, false, false>(d, s, logits, ws, st);
  hipLaunchKernelGGL((distill_finish_kernel<Ty>), dim3(d.T), dim3(64), 0, st, finish_args(d, s.S),
                     static_cast<const typename Ty::E*>(logits), idx, teacher, reinterpret_cast<const float4*>(ws), loss,
                     stats);
}

template <class Ty>
void logprobs_bwd_launch(const VocabDims& d, const LogprobGradPtrs& q, hipStream_t st) {
  const BwdArgs b = bwd_args(d);
  auto* f = d.accumulate ? logprobs_bwd_kernel<Ty, true> : logprobs_bwd_kernel<Ty, false>;
  hipLaunchKernelGGL(f, dim3((size_t)d.T * b.S), dim3(256), 0, st, b, q);
}

template <class Ty>
void distill_bwd_launch(const VocabDims& d, const void* logits, const int* idx, const float* teacher,
                        const float* stats, const float* g_loss, void* d_logits, hipStream_t st) {
  typedef typename Ty::E E;
  const BwdArgs b = bwd_args(d);
  auto* f = d.accumulate ? distill_bwd_kernel<Ty, true> : distill_bwd_kernel<Ty, false>;
  hipLaunchKernelGGL(f, dim3((size_t)d.T * b.S), dim3(256), 0, st, b, static_cast<const E*>(logits), idx, teacher,
                     stats, g_loss, static_cast<E*>(d_logits));
}

}  // namespace

size_t vocab_ws_bytes(const VocabDims& d) {
  return part_bytes(d) + (d.k > 0 ? (size_t)d.T * blocks_of(d.V) * (d.f32 ? 4 : 2) : 0);
}

hipError_t launch_token_logprobs(const VocabDims& d, const LogprobPtrs& q, char* ws, hipStream_t st) {
  ProfScope prof(st, "vocab.logprobs");
  d.f32 ? logprobs_launch<F32>(d, q, ws, st) : logprobs_launch<Bf16>(d, q, ws, st);
  return hipGetLastError();
}

hipError_t launch_token_logprobs_bwd(const VocabDims& d, const LogprobGradPtrs& q, hipStream_t st) {
  ProfScope prof(st, "vocab.logprobs_bwd");
  d.f32 ? logprobs_bwd_launch<F32>(d, q, st) : logprobs_bwd_launch<Bf16>(d, q, st);
  return hipGetLastError();
}

hipError_t launch_distill(const VocabDims& d, const void* logits, const int* idx, const float* teacher, float* loss,
                          float* stats, char* ws, hipStream_t st) {
  ProfScope prof(st, "vocab.distill");
  d.f32 ? distill_launch<F32>(d, logits, idx, teacher, loss, stats, ws, st)
        : distill_launch<Bf16>(d, logits, idx, teacher, loss, stats, ws, st);
  return hipGetLastError();
}

hipError_t launch_distill_bwd(const VocabDims& d, const void* logits, const int* idx, const float* teacher,
                              const float* stats, const float* g_loss, void* d_logits, hipStream_t st) {
  ProfScope prof(st, "vocab.distill_bwd");
  d.f32 ? distill_bwd_launch<F32>(d, logits, idx, teacher, stats, g_loss, d_logits, st)
        : distill_bwd_launch<Bf16>(d, logits, idx, teacher, stats, g_loss, d_logits, st);
  return hipGetLastError();
}

}  // namespace oft
