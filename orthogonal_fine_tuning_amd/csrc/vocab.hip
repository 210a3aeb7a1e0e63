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

// value of another lane of the same 16 (DPP)
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
constexpr int PAIR = 0xB1, QUAD = 0x4E, EIGHT = 0x141, ROW = 0x140;  // lanes ^ 1, ^ 2, 7 - i of 8, 15 - i of 16
__device__ __forceinline__ float lane_value(float v, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}
// over the wave's 64 lanes (all active), the same bits in every lane
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<PAIR>(v);
  v += dpp<QUAD>(v);
  v += dpp<EIGHT>(v);
  v += dpp<ROW>(v);
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp<PAIR>(v));
  v = fmaxf(v, dpp<QUAD>(v));
  v = fmaxf(v, dpp<EIGHT>(v));
  v = fmaxf(v, dpp<ROW>(v));
  return fmaxf(fmaxf(lane_value(v, 0), lane_value(v, 16)), fmaxf(lane_value(v, 32), lane_value(v, 48)));
}

// ------------------------------------------------------------------ triples
struct Triple {
  float m, s, w;
};

// the triple moved to the maximum M >= m; an empty set has s = 0
__device__ __forceinline__ Triple moved(const Triple& a, float M, float c) {
  const float d = a.s == 0.0f ? 0.0f : a.m - M;
  const float f = exp2_hw(c * d);
  return Triple{M, a.s * f, f * fmaf(a.s, fmaxf(d, FAR), a.w)};
}

__device__ __forceinline__ Triple join(const Triple& a, const Triple& b, float c) {
  const float M = fmaxf(a.m, b.m);
  const Triple x = moved(a, M, c), y = moved(b, M, c);
  return Triple{M, x.s + y.s, x.w + y.w};
}

__device__ __forceinline__ Triple wave_join(const Triple& a, float c) {
  const float M = wave_max(a.m);
  const Triple x = moved(a, M, c);
  return Triple{M, wave_sum(x.s), wave_sum(x.w)};
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
  a = moved(a, fmaxf(a.m, bm), c);
  const float ref = a.m == -INFINITY ? 0.0f : a.m;
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
      float v = fmaxf(vm[u], dpp<PAIR>(vm[u]));
      v = fmaxf(v, dpp<QUAD>(v));
      v = fmaxf(v, dpp<EIGHT>(v));
      if constexpr (G == 16) v = fmaxf(v, dpp<ROW>(v));
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

// ---------------------------------------------------------- top alternatives
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

template <class Ty>
__device__ __forceinline__ float rank_value(typename Ty::E v) {  // NaN ranks as -inf
  const float f = Ty::get(v);
  return f != f ? -INFINITY : f;
}

// k-th largest of the N lane values (in `ordered` form), two bits a step.
// Values of 16 bits (LOW = 16) are told apart by their upper half.
template <int N, int LOW>
__device__ __forceinline__ uint32_t kth(const uint32_t (&o)[N], int k) {
  uint32_t r = 0;
  for (int bit = 30; bit >= LOW; bit -= 2) {
    int n1 = 0, n2 = 0, n3 = 0;
    const uint32_t t1 = r | (1u << bit), t2 = r | (2u << bit), t3 = r | (3u << bit);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      n1 += __popcll(__ballot(o[j] >= t1));
      n2 += __popcll(__ballot(o[j] >= t2));
      n3 += __popcll(__ballot(o[j] >= t3));
    }
    r = n3 >= k ? t3 : n2 >= k ? t2 : n1 >= k ? t1 : r;
  }
  return r;
}

// LDS of one wave, written and read by its lanes
__device__ __forceinline__ void wave_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A wave's selection of the k best of a stream of (value, id), ids ascending:
// candidates wait in LDS in order of id; when the list is full it is cut to
// its k best, whose last value is then what a later candidate must exceed.
// Right for any input, whatever its ties.
constexpr int QCAP = 512, MAXTOP = 128;
struct Select {
  float* val;  // [QCAP] in LDS
  int* id;     // [QCAP]
  int k, n;
  float floor;  // a candidate must reach it, or exceed it once `strict`
  bool strict;

  __device__ __forceinline__ Select(float* v, int* i, int kk, float f)
      : val(v), id(i), k(kk), n(0), floor(f), strict(false) {}

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
    wave_lds();
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
    const uint32_t last = kth<N, 0>(o, k);
    int above = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) above += __popcll(__ballot(o[j] > last));
    int ties = k - above, m = 0;
    wave_lds();
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const bool tie = o[j] == last && j * 64 + lane < n;
      const unsigned long long eq = __ballot(tie);
      const bool keep = o[j] > last || (tie && below(eq) < ties);
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
    wave_lds();
  }
};

struct FinishArgs {
  int V, k, S, nb;
  long ld;
  float c, invtau;
};

// Top alternatives of a row by one wave: the k best blocks, then the k best of
// their elements.  val, id: [2][QCAP]; the result is val[1], id[1] in order
// of column, at least k of them.
template <class Ty>
__device__ void select_any(const FinishArgs& f, const typename Ty::E* row, const typename Ty::E* brow,
                           float (*val)[QCAP], int (*id)[QCAP]) {
  constexpr int U = 8;  // loads in flight
  const int lane = threadIdx.x & 63;
  // a value that at least k blocks reach: the k-th best of 128 interleaved
  // groups of blocks
  float best[2] = {-INFINITY, -INFINITY};
  for (int b = lane; b < f.nb; b += 64 * U) {
#pragma unroll
    for (int j = 0; j < U; ++j)
      if (b + 64 * j < f.nb) best[j & 1] = fmaxf(best[j & 1], Ty::get(brow[b + 64 * j]));
  }
  const uint32_t o[2] = {ordered(best[0]), ordered(best[1])};
  Select sel(val[0], id[0], f.k, unordered(kth<2, 0>(o, f.k)));
  for (int b = lane; b - lane < f.nb; b += 64 * U) {
    float v[U];
#pragma unroll
    for (int j = 0; j < U; ++j) v[j] = b + 64 * j < f.nb ? rank_value<Ty>(brow[b + 64 * j]) : 0.0f;
#pragma unroll
    for (int j = 0; j < U; ++j) sel.feed(v[j], b + 64 * j, b + 64 * j < f.nb);
  }
  sel.cut();
  // the blocks' elements: at least k reach the least of k maxima
  const int nsel = sel.n;
  float lowest = INFINITY;
  for (int i = lane; i < nsel; i += 64) lowest = fminf(lowest, val[0][i]);
  lowest = -wave_max(-lowest);
  Select el(val[1], id[1], f.k, nsel < f.k ? -INFINITY : lowest);
  for (int i = 0; i < nsel; i += U) {
    float v[U];
    int col[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      col[j] = i + j < nsel ? id[0][i + j] * BLOCK + lane : f.V;
      v[j] = col[j] < f.V ? rank_value<Ty>(row[col[j]]) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < U; ++j) el.feed(v[j], col[j], col[j] < f.V);
  }
  el.cut();
}

// Joins a row's slices; its outputs.  Four waves per row.
//
// Top alternatives, the usual case: each thread holds up to HELD block maxima
// in registers; a value T that k of 256 (k <= 64) or 512 disjoint groups of
// them reach is at most the k-th best, so the elements >= T of the blocks
// >= T hold the answer.  There are few more than k of them, in any order:
// (value, column) as one 64-bit key gives each its place by counting the
// keys above it.  Rows where ties or masks leave too many (or a vocabulary of
// more blocks than the registers hold) go through select_any.
constexpr int HELD = 16, MAXBLK = 512, MAXCAND = 512;
template <class Ty, bool TOP>
__global__ __launch_bounds__(256) void logprobs_finish_kernel(FinishArgs f, LogprobPtrs q,
                                                              const float4* __restrict__ part,
                                                              const typename Ty::E* __restrict__ blocks) {
  typedef typename Ty::E E;
  const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
  const E* row = static_cast<const E*>(q.logits) + (size_t)t * f.ld;
  const E* brow = TOP ? blocks + (size_t)t * f.nb : nullptr;
  float held[HELD];
  const bool few = f.nb <= HELD * 256;
  if constexpr (TOP) {
#pragma unroll
    for (int i = 0; i < HELD; ++i) held[i] = few && i * 256 + tid < f.nb ? rank_value<Ty>(brow[i * 256 + tid]) : NAN;
  }
  const int lab = q.logp && tid == 0 ? q.labels[t] : -1;
  const bool known = lab >= 0 && lab < f.V;
  const float given = known ? Ty::get(row[lab]) : 0.0f;
  Triple a{-INFINITY, 0.0f, 0.0f};
  for (int i = lane; i < f.S; i += 64) {
    const float4 p = part[(size_t)t * f.S + i];
    a = join(a, Triple{p.x, p.y, p.z}, f.c);
  }
  a = wave_join(a, f.c);
  const bool empty = a.s == 0.0f;
  const float l = __logf(a.s);  // ln 0 = -inf for an empty row
  if (tid == 0) {
    *reinterpret_cast<float2*>(q.stats + 2 * (size_t)t) = make_float2(a.m, l);
    if (q.entropy) q.entropy[t] = empty ? 0.0f : l - a.w * f.invtau / a.s;
    if (q.logp)
      q.logp[t] = lab == -1 ? 0.0f : !known ? NAN : empty ? -INFINITY : (given - a.m) * f.invtau - l;
  }
  if constexpr (TOP) {
    constexpr int LOW = sizeof(E) == 2 ? 16 : 0;
    __shared__ __align__(16) unsigned long long key[MAXCAND];
    __shared__ float val[2][QCAP];
    __shared__ int id[2][QCAP];
    __shared__ uint32_t group[512];
    __shared__ int cand_block[MAXBLK];
    __shared__ float sh_floor;
    __shared__ int nblk, ncand;
    if (tid == 0) nblk = ncand = 0;
    float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < HELD; ++i) best[i & 1] = fmaxf(best[i & 1], held[i]);
    group[tid] = ordered(f.k <= 64 ? fmaxf(best[0], best[1]) : best[0]);
    if (f.k > 64) group[256 + tid] = ordered(best[1]);
    __syncthreads();
    if (tid < 64) {
      uint32_t r;
      if (f.k <= 64) {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = group[64 * j + lane];
        r = kth<4, LOW>(o, f.k);
      } else {
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = group[64 * j + lane];
        r = kth<8, LOW>(o, f.k);
      }
      // (of a negative 16-bit value the lower half of the ordered form is ones)
      if (tid == 0) sh_floor = r == 0u ? -INFINITY : unordered(LOW && !(r & 0x80000000u) ? r | 0xFFFFu : r);
    }
    __syncthreads();
    const float floor = sh_floor;
#pragma unroll
    for (int i = 0; i < HELD; ++i)
      if (held[i] >= floor) {  // (false for NaN: no block)
        const int at = atomicAdd(&nblk, 1);
        if (at < MAXBLK) cand_block[at] = i * 256 + tid;
      }
    __syncthreads();
    const int n1 = nblk;
    bool usual = few && n1 <= MAXBLK;
    if (usual) {
      constexpr int U = 8;
      for (int i = tid >> 6; i < n1; i += 4 * U) {
        float v[U];
        int col[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
          col[j] = i + 4 * j < n1 ? cand_block[i + 4 * j] * BLOCK + lane : f.V;
          v[j] = col[j] < f.V ? rank_value<Ty>(row[col[j]]) : NAN;
        }
#pragma unroll
        for (int j = 0; j < U; ++j)
          if (v[j] >= floor) {
            const int at = atomicAdd(&ncand, 1);
            if (at < MAXCAND) key[at] = (unsigned long long)ordered(v[j]) << 32 | (uint32_t)~col[j];
          }
      }
      __syncthreads();
      usual = ncand <= MAXCAND;
    }
    int n = usual ? ncand : f.k;
    if (!usual) {
      __syncthreads();
      if (tid < 64) {
        select_any<Ty>(f, row, brow, val, id);
        for (int i = lane; i < f.k; i += 64)
          key[i] = (unsigned long long)ordered(val[1][i]) << 32 | (uint32_t)~id[1][i];
      }
      __syncthreads();
    }
    // an even number of keys for the paired reads: 0 is below every key
    if (tid == 0 && (n & 1)) key[n] = 0ull;
    __syncthreads();
    for (int i = tid; i < n; i += 256) {
      const unsigned long long mine = key[i];
      int place = 0;
      for (int j = 0; j < n; j += 2) {
        const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(key + j);
        place += (o.x > mine ? 1 : 0) + (o.y > mine ? 1 : 0);
      }
      if (place < f.k) {
        const float v = unordered((uint32_t)(mine >> 32));
        const size_t at = (size_t)t * f.k + place;
        q.top_idx[at] = (int)~(uint32_t)mine;
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
    mx = wave_max(mx);
    any = mx != -INFINITY;
    float s = 0.0f, e[TI];
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      logq[i] = any ? (v[i] - mx) * invtau : -INFINITY;
      e[i] = exp2_hw(logq[i] * LOG2E);
      s += e[i];
    }
    s = wave_sum(s);
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
  Triple a{-INFINITY, 0.0f, 0.0f};
  for (int i = threadIdx.x; i < f.S; i += 64) {
    const float4 p = part[(size_t)t * f.S + i];
    a = join(a, Triple{p.x, p.y, p.z}, f.c);
  }
  a = wave_join(a, f.c);
  const float l = __logf(a.s);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < TI; ++i)
    if (te.ix[i] >= 0) {
      const float lp = a.s == 0.0f ? -INFINITY : (x[i] - a.m) * f.invtau - l;
      sum = fmaf(te.q[i], te.logq[i] - lp, sum);
    }
  sum = wave_sum(sum);
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
      grad(x, i0);
#pragma unroll
      for (int j = 0; j < VE; ++j) x[j] += ACC ? o[j] : 0.0f;
      store16(out + i0, Ty::pack(x));
    }
  }
  for (int i0 = base + tid * VE; i0 < hi; i0 += 256 * VE) {
    float x[VE], o[VE];
    if (i0 + VE <= hi) {
      Ty::unpack(load16(row + i0), x);
      if constexpr (ACC) Ty::unpack(load16(out + i0), o);
      grad(x, i0);
#pragma unroll
      for (int j = 0; j < VE; ++j) x[j] += ACC ? o[j] : 0.0f;
      store16(out + i0, Ty::pack(x));
    } else {
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        x[j] = i0 + j < hi ? Ty::get(row[i0 + j]) : 0.0f;
        o[j] = ACC && i0 + j < hi ? Ty::get(out[i0 + j]) : 0.0f;
      }
      grad(x, i0);
#pragma unroll
      for (int j = 0; j < VE; ++j)
        if (i0 + j < hi) out[i0 + j] = Ty::put(x[j] + o[j]);
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
  bwd_columns<Ty, ACC>(row, out, lo, hi, fill, [&](float (&x)[Ty::VE], int i0) {
#pragma unroll
    for (int j = 0; j < Ty::VE; ++j) x[j] = g(x[j]);
    if ((unsigned)(lab - i0) < (unsigned)Ty::VE) {
#pragma unroll
      for (int j = 0; j < Ty::VE; ++j) x[j] += lab - i0 == j ? at : 0.0f;
    }
  });
}

template <class Ty, bool ACC>
__global__ __launch_bounds__(256) void distill_bwd_kernel(BwdArgs b, const typename Ty::E* logits,
                                                          const int* __restrict__ idx,
                                                          const float* __restrict__ teacher,
                                                          const float* __restrict__ stats,
                                                          const float* __restrict__ g_loss, typename Ty::E* d_logits) {
  typedef typename Ty::E E;
  __shared__ __align__(16) int lidx[64 * TI + 4];
  __shared__ __align__(16) float lq[64 * TI + 4];
  const int t = blockIdx.x / b.S, sl = blockIdx.x % b.S, tid = threadIdx.x;
  const E* row = logits + (size_t)t * b.ld;
  E* out = d_logits + (size_t)t * b.ldg;
  const int lo = sl * b.slice, hi = min(b.V, lo + b.slice);
  const float2 st = *reinterpret_cast<const float2*>(stats + 2 * (size_t)t);
  const float g = g_loss[t];
  // (each wave computes the list; all get the same)
  const Teacher te(idx + (size_t)t * b.k, teacher + (size_t)t * b.k, b.k, b.V, b.invtau);
  int fill = FILL_NONE;
  if (g == 0.0f) fill = FILL_ZERO;
  else if (te.bad) fill = FILL_NAN;
  else if (!te.any || st.y == -INFINITY) fill = FILL_ZERO;
  const RowGrad r{st.x, b.c, st.y * LOG2E, 0.0f, g * b.invtau};
  // the entries of this slice, in list order
  int n = 0;
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const bool in = te.ix[i] >= lo && te.ix[i] < hi;
    const unsigned long long mask = __ballot(in);
    if (in && tid < 64) {
      lidx[n + below(mask)] = te.ix[i];
      lq[n + below(mask)] = te.q[i];
    }
    n += __popcll(mask);
  }
  if (tid < 4) lidx[n + tid] = -1;  // up to a multiple of four
  __syncthreads();
  // one entry per thread: the column's gradient p - sum of its q.  Read
  // before anything is written (d_logits may be logits)
  const bool listed = fill == FILL_NONE && tid < n;
  const int mine = listed ? lidx[tid] : 0;
  float v = 0.0f;
  if (listed) {
    v = exp2_hw(r.log2p(Ty::get(row[mine])));
    float q = 0.0f;
    for (int j = 0; j < n; j += 4) {
      const int4 li = *reinterpret_cast<const int4*>(lidx + j);
      const float4 qi = *reinterpret_cast<const float4*>(lq + j);
      q += li.x == mine ? qi.x : 0.0f;
      q += li.y == mine ? qi.y : 0.0f;
      q += li.z == mine ? qi.z : 0.0f;
      q += li.w == mine ? qi.w : 0.0f;
    }
    v = (v - q) * r.gb;
    if constexpr (ACC) v += Ty::get(out[mine]);
  }
  __syncthreads();
  bwd_columns<Ty, ACC>(row, out, lo, hi, fill, [&](float (&x)[Ty::VE], int) {
#pragma unroll
    for (int j = 0; j < Ty::VE; ++j) x[j] = exp2_hw(r.log2p(x[j])) * r.gb;
  });
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
    hipLaunchKernelGGL((logprobs_finish_kernel<Ty, true>), dim3(d.T), dim3(256), 0, st, f, q, part, blocks);
  } else {
    if (q.entropy) stats_launch<Ty, true, false>(d, s, q.logits, ws, st);
    else stats_launch<Ty, false, false>(d, s, q.logits, ws, st);
    hipLaunchKernelGGL((logprobs_finish_kernel<Ty, false>), dim3(d.T), dim3(256), 0, st, f, q, part, blocks);
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
