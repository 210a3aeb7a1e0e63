// Losses on vocabulary logits (include/oft.h): log-probabilities of given
// tokens with entropy and top alternatives, distillation from a teacher's
// top logits, and their gradients.
//
// With x a row, m its maximum, c = log2(e) / tau and R = c m as rounded:
//   e_i = 2^(c x_i - R) (one fused multiply-add, so its rounding is relative
//   to the small difference, and R is a reference like any other),
//   s = sum e_i, w = sum e_i (c x_i - R),
//   l = ln s - (c m - R) ln 2, H = (log2 s - w / s) ln 2,
//   log p_i = (x_i - m) / tau - l.
// A sum over part of a row is the triple (m, s, w) with its own m; moving it
// to a larger maximum multiplies s by f = 2^d, d the difference of the two
// references, and turns w into f (w + s d).
//
// Forward: every logit is read once, which bounds large calls (4096 x 151936
// bf16: 187 us for the distillation loss, 6.7 TB/s; 198 us with entropy and 20
// alternatives).  A workgroup takes a whole row (logprobs_row_kernel,
// distill_row_kernel), or a slice of one where rows are few:
// vocab_stats_kernel leaves a triple per slice, logprobs_finish_kernel and
// distill_finish_kernel join them.  For the top alternatives the pass also
// keeps the maximum of every block of 64 columns: any value that k blocks
// reach is at most the k-th best logit, so only the blocks that reach such a
// value are read again.
//
// Backward: one read and one write per logit with (m, l) from the forward
// (4096 x 151936 bf16: 390 us, 6.2 TB/s both ways).
//
// Rows start anywhere: gfx950 takes 16-byte loads at any 4-byte address at full
// speed (at 2-byte ones 30 % slower, 126 for 96 us at 2048 x 151935 bf16).  So
// a bf16 row at an odd element is taken from one element earlier: positions
// are columns + skew, and position 0 is no column.  Only a row's partial
// vectors are read by elements, so nothing outside a row is touched.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "oft_device.h"
#include "oft_launch.h"
#include "oft_prof.h"
#include "oft_vocab.h"

namespace oft {
namespace {

constexpr float LOG2E = 1.44269504088896340736f;
constexpr float LN2 = 0.69314718055994530942f;
// clamp of base-2 exponents where they meet their own 2^x: that is 0 in fp32
// far above it, and 0 times it is 0 (0 times -inf would be NaN)
constexpr float LOWEST = -1000.0f;
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
// a vector that is read or written once; NT: it need not displace what the
// caches hold (STREAM_BYTES below)
template <bool NT, class E>
__device__ __forceinline__ u32x4 stream16(const E* p) {
  const u32x4_row* v = reinterpret_cast<const u32x4_row*>(p);
  return NT ? __builtin_nontemporal_load(v) : *v;
}
template <bool NT, class E>
__device__ __forceinline__ void stream16(E* p, const u32x4& v) {
  if constexpr (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_row*>(p));
  else *reinterpret_cast<u32x4_row*>(p) = v;
}

// elements that a row is taken early
template <class Ty>
__device__ __forceinline__ int skew_of(const typename Ty::E* row) {
  return sizeof(typename Ty::E) == 2 ? (int)(reinterpret_cast<uintptr_t>(row) >> 1 & 1) : 0;
}

// value of another lane of the same 16 (DPP)
template <int CTRL, class T>
__device__ __forceinline__ T dpp(T v) {
  return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
constexpr int PAIR = 0xB1, QUAD = 0x4E, EIGHT = 0x141, ROW = 0x140;  // lanes ^ 1, ^ 2, 7 - i of 8, 15 - i of 16
template <class T>
__device__ __forceinline__ T lane_value(T v, int l) {
  return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}
// over the wave's 64 lanes (all active), the same bits in every lane
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
  v += dpp<PAIR>(v);
  v += dpp<QUAD>(v);
  v += dpp<EIGHT>(v);
  v += dpp<ROW>(v);
  return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
template <class T>
__device__ __forceinline__ T wave_max(T v) {
  v = larger(v, dpp<PAIR>(v));
  v = larger(v, dpp<QUAD>(v));
  v = larger(v, dpp<EIGHT>(v));
  v = larger(v, dpp<ROW>(v));
  return larger(larger(lane_value(v, 0), lane_value(v, 16)), larger(lane_value(v, 32), lane_value(v, 48)));
}

// LDS of one wave, written and read by its lanes
__device__ __forceinline__ void wave_lds() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ------------------------------------------------------------------ triples
struct Triple {
  float m, s, w;
};

// R of a maximum; 0 for an empty set.  From 2^20 on, where the rounding of
// c m is no longer small against 1 (masks at the type's lowest value alone in
// a part of a row), the reference is c m itself: 2^(c (x - m)).
__device__ __forceinline__ float reference(float m, float c) { return m == -INFINITY ? 0.0f : c * m; }
__device__ __forceinline__ bool beyond(float R) { return !(fabsf(R) < 0x1p20f); }
// c m less the reference
__device__ __forceinline__ float rounding(float m, float R, float c) {
  return m == -INFINITY || beyond(R) ? 0.0f : fmaf(c, m, -R);
}

// the triple moved to the maximum M >= m; an empty set has s = 0
__device__ __forceinline__ Triple moved(const Triple& a, float M, float c) {
  const float Ra = reference(a.m, c), RM = reference(M, c);
  float d = beyond(Ra) || beyond(RM) ? c * (a.m - M) + (rounding(M, RM, c) - rounding(a.m, Ra, c)) : Ra - RM;
  d = a.s == 0.0f ? 0.0f : d;
  const float f = exp2_hw(d);
  return Triple{M, a.s * f, f * fmaf(a.s, fmaxf(d, LOWEST), a.w)};
}

// l of a row's triple: -inf for an empty row
__device__ __forceinline__ float log_sum(const Triple& a, float c) {
  return (__builtin_amdgcn_logf(a.s) - rounding(a.m, reference(a.m, c), c)) * LN2;
}
__device__ __forceinline__ float entropy_of(const Triple& a) {
  return a.s == 0.0f ? 0.0f : (__builtin_amdgcn_logf(a.s) - a.w / a.s) * LN2;
}

// k (x - m), also where the difference of finite values alone passes fp32's
// range (for x = -inf the two products could be infinite alike)
__device__ __forceinline__ float scaled(float x, float m, float k) {
  const float d = x - m;
  return d == -INFINITY && x > -INFINITY ? k * x - k * m : k * d;
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

// Order of the top alternatives as an unsigned number: larger value first,
// -0 as +0, NaN as -inf.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, (v == v ? v : -INFINITY) + 0.0f);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __builtin_bit_cast(float, (o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}

// Block maxima of a row, as `ordered` numbers: the upper half of it says all
// for bf16.  A block is 64 columns of one step of the forward pass: the 64 / FU
// columns of each of its FU vectors that RUN neighbouring lanes hold.
template <class Ty>
struct Blocks {
  typedef std::conditional_t<sizeof(typename Ty::E) == 2, uint16_t, uint32_t> Key;
  static constexpr int BITS = 8 * sizeof(Key);
  static constexpr int RUN = 64 / FU / Ty::VE;            // lanes
  static constexpr int PER_TILE = 256 / RUN;              // blocks of a step
  static constexpr int VECS = FU * RUN;                   // 16-byte vectors of a block
  static constexpr int TILE = fwd_tile<Ty>();
  static __device__ __forceinline__ uint32_t key(float v) { return ordered(v) >> (32 - BITS); }
  // first position of vector i of block b
  static __device__ __forceinline__ int position(int b, int i) {
    return b / PER_TILE * TILE + i / RUN * (256 * Ty::VE) + b % PER_TILE * (64 / FU) + i % RUN * Ty::VE;
  }
};

// a block's maximum, from its lanes' own maxima
template <class Ty>
__device__ __forceinline__ typename Blocks<Ty>::Key block_key(float v) {
  if constexpr (Blocks<Ty>::RUN >= 2) v = fmaxf(v, dpp<PAIR>(v));
  if constexpr (Blocks<Ty>::RUN == 4) v = fmaxf(v, dpp<QUAD>(v));
  return (typename Blocks<Ty>::Key)Blocks<Ty>::key(v);
}

// What becomes of the block maxima of a workgroup's steps.
// Nothing:
struct KeepNone {
  __device__ __forceinline__ void add(float) {}
  __device__ __forceinline__ void flush() {}
};
// they stay in LDS, the whole row's:
template <class Ty>
struct KeepRow {
  typedef typename Blocks<Ty>::Key Key;
  Key* lds;  // the next step's PER_TILE keys
  __device__ __forceinline__ void add(float v) {
    const Key k = block_key<Ty>(v);
    if (threadIdx.x % Blocks<Ty>::RUN == 0) lds[threadIdx.x / Blocks<Ty>::RUN] = k;
    lds += Blocks<Ty>::PER_TILE;
  }
  __device__ __forceinline__ void flush() {}
};
// or they go to memory: a wave's keys of KEPT steps, 64 bytes each, wait in
// LDS and leave as one 16-byte store per lane
constexpr int KEPT = 16;
template <class Ty>
struct KeepOut {
  typedef typename Blocks<Ty>::Key Key;
  static constexpr int PW = 64 / Blocks<Ty>::RUN, PV = 16 / sizeof(Key);  // keys of a wave's step, of a vector
  static_assert(PW == 4 * PV, "four vectors a step");
  Key* lds;  // this wave's [KEPT][PW]
  Key* out;  // this wave's first key of the first step kept
  int n;     // steps kept

  __device__ __forceinline__ void add(float v) {
    const Key k = block_key<Ty>(v);
    const int lane = threadIdx.x & 63;
    if (lane % Blocks<Ty>::RUN == 0) lds[n * PW + lane / Blocks<Ty>::RUN] = k;
    if (++n == KEPT) flush();
  }
  __device__ __forceinline__ void flush() {
    wave_lds();
    const int step = (threadIdx.x & 63) / 4, part = threadIdx.x % 4;
    if (step < n)
      *reinterpret_cast<u32x4*>(out + step * Blocks<Ty>::PER_TILE + part * PV) =
          *reinterpret_cast<const u32x4*>(lds + step * PW + part * PV);
    wave_lds();
    out += n * Blocks<Ty>::PER_TILE;
    n = 0;
  }
};

// one step: FU vectors per thread, x[u VE + j] is position base + (u 256 + tid)
// VE + j; again(u, y) reads vector u once more.  Returns the thread's maximum.
template <class Ty, bool ENT, class F>
__device__ __forceinline__ float fwd_step(const float (&x)[FU * Ty::VE], float c, Triple& a, F again) {
  constexpr int N = FU * Ty::VE;
  float m0 = x[0], m1 = x[1];
#pragma unroll
  for (int i = 2; i < N; i += 4) {
    m0 = fmaxf(fmaxf(m0, x[i]), x[i + 1]);
    if (i + 2 < N) m1 = fmaxf(fmaxf(m1, x[i + 2]), x[i + 3]);
  }
  const float bm = fmaxf(m0, m1);
  a = moved(a, fmaxf(a.m, bm), c);
  const float R = reference(a.m, c);
  float s[2] = {0.0f, 0.0f}, w[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float z = fmaf(x[i], c, -R);
    const float e = exp2_hw(z);
    s[i & 1] += e;
    if constexpr (ENT) w[i & 1] = fmaf(e, z, w[i & 1]);
  }
  float sum = s[0] + s[1], sumw = w[0] + w[1];
  // (the sums stay on this side of the branch: their terms would hold registers)
  asm volatile("" : "+v"(sum), "+v"(sumw));
  // Some lane has a masked logit (0 * -inf in w) or a far reference:
  // the wave's step once more with neither, from a second read, so that steps
  // without them are spared the instructions and x need not outlive its sums.
  if (__ballot((ENT && sumw != sumw) || beyond(R)) != 0) {
    // (in the same order, so that l does not depend on whether H is wanted)
    s[0] = s[1] = w[0] = w[1] = 0.0f;
#pragma unroll 1
    for (int u = 0; u < FU; ++u) {
      float y[Ty::VE];
      again(u, y);
#pragma unroll
      for (int j = 0; j < Ty::VE; ++j) {
        const float z = beyond(R) ? c * (y[j] - a.m) : fmaf(y[j], c, -R);
        const float e = exp2_hw(z);
        s[j & 1] += e;
        w[j & 1] = fmaf(e, fmaxf(z, LOWEST), w[j & 1]);
      }
    }
    sum = s[0] + s[1];
    sumw = w[0] + w[1];
  }
  a.s += sum;
  a.w += sumw;
  return bm;
}

// one vector, with masked logits and any reference: a row's last, partial step
template <class Ty, bool ENT>
__device__ __forceinline__ float fwd_vector(const float* x, float c, Triple& a) {
  float bm = x[0];
#pragma unroll
  for (int j = 1; j < Ty::VE; ++j) bm = fmaxf(bm, x[j]);
  a = moved(a, fmaxf(a.m, bm), c);
  const float R = reference(a.m, c);
  const bool far = beyond(R);
#pragma unroll
  for (int j = 0; j < Ty::VE; ++j) {
    const float z = far ? c * (x[j] - a.m) : fmaf(x[j], c, -R);
    const float e = exp2_hw(z);
    a.s += e;
    if constexpr (ENT) a.w = fmaf(e, fmaxf(z, LOWEST), a.w);
  }
  return bm;
}

// vector at position i0 of a row's positions [skew, hi), -inf elsewhere; `row`
// is where position 0 would be
template <class Ty, bool NT>
__device__ __forceinline__ void read_vector(const typename Ty::E* row, int i0, int skew, int hi, float* y) {
  constexpr int VE = Ty::VE;
  if (i0 >= skew && i0 + VE <= hi) {
    Ty::unpack(stream16<NT>(row + i0), y);
  } else {
#pragma unroll
    for (int j = 0; j < VE; ++j) y[j] = i0 + j >= skew && i0 + j < hi ? Ty::get(row[i0 + j]) : -INFINITY;
  }
}

// The triple of positions [lo, hi) of a row by a workgroup, the same in every
// thread; lo starts a step.
template <class Ty, bool ENT, bool NT, class K>
__device__ __forceinline__ Triple slice_triple(const typename Ty::E* row, int skew, int lo, int hi, float c, K& keep) {
  constexpr int VE = Ty::VE, TILE = fwd_tile<Ty>();
  __shared__ float sh[4][3];
  const int tid = threadIdx.x;
  Triple a{-INFINITY, 0.0f, 0.0f};
  float x[FU * VE];
  int base = lo;
  u32x4 v[FU];
  if (base + TILE <= hi) {
#pragma unroll
    for (int u = 0; u < FU; ++u)
      if (u > 0 || lo + tid > 0 || skew == 0) v[u] = stream16<NT>(row + base + (u * 256 + tid) * VE);
    if (skew != 0 && lo + tid == 0) {  // position 0 is no column: -inf before the row's first seven
      const u32x4 f = load16(row + 1);
      v[0] = u32x4{f[0] << 16 | 0xFF80u, f[1] << 16 | f[0] >> 16, f[2] << 16 | f[1] >> 16, f[3] << 16 | f[2] >> 16};
    }
  }
  for (; base + TILE <= hi; base += TILE) {
#pragma unroll
    for (int u = 0; u < FU; ++u) Ty::unpack(v[u], x + u * VE);
    // the next step's loads fly during this one's sums
    if (base + 2 * TILE <= hi) {
#pragma unroll
      for (int u = 0; u < FU; ++u) v[u] = stream16<NT>(row + base + TILE + (u * 256 + tid) * VE);
    }
    keep.add(fwd_step<Ty, ENT>(
        x, c, a, [&](int u, float* y) { read_vector<Ty, NT>(row, base + (u * 256 + tid) * VE, skew, hi, y); }));
  }
  if (base < hi) {
#pragma unroll
    for (int u = 0; u < FU; ++u) read_vector<Ty, NT>(row, base + (u * 256 + tid) * VE, skew, hi, x + u * VE);
    float bm = -INFINITY;
#pragma unroll
    for (int u = 0; u < FU; ++u)
      if (base + (u * 256 + (tid & ~63)) * VE < hi) bm = fmaxf(bm, fwd_vector<Ty, ENT>(x + u * VE, c, a));
    keep.add(bm);
  }
  keep.flush();
  a = wave_join(a, c);
  if ((tid & 63) == 0) {
    sh[tid >> 6][0] = a.m;
    sh[tid >> 6][1] = a.s;
    sh[tid >> 6][2] = a.w;
  }
  __syncthreads();
  a = Triple{sh[0][0], sh[0][1], sh[0][2]};
#pragma unroll
  for (int i = 1; i < 4; ++i) a = join(a, Triple{sh[i][0], sh[i][1], sh[i][2]}, c);
  return a;
}

// part[t S + sl]: the triple of positions [sl slice, (sl + 1) slice) of row t;
// blocks: the maxima of the row's blocks, rows of them nb apart.  (One row of
// 151936 bf16 columns, 19 slices: 4.4 us; 64 rows 7.6 us.)
template <class Ty, bool ENT, bool TOP, bool NT>
__global__ __launch_bounds__(256) void vocab_stats_kernel(const typename Ty::E* __restrict__ logits, long ld, int V,
                                                          int S, int slice, float c, float4* __restrict__ part,
                                                          typename Blocks<Ty>::Key* __restrict__ blocks, int nb) {
  typedef Blocks<Ty> B;
  typedef typename B::Key Key;
  const int t = blockIdx.x / S, sl = blockIdx.x % S, tid = threadIdx.x;
  const typename Ty::E* row = logits + (size_t)t * ld;
  const int skew = skew_of<Ty>(row);
  row -= skew;
  const int lo = sl * slice, hi = min(V + skew, lo + slice);
  Triple a;
  if constexpr (TOP) {
    __shared__ __align__(16) Key kept[4][KEPT * KeepOut<Ty>::PW];
    KeepOut<Ty> keep{kept[tid >> 6],
                     blocks + (size_t)t * nb + lo / fwd_tile<Ty>() * B::PER_TILE + (tid & ~63) / B::RUN, 0};
    a = slice_triple<Ty, ENT, NT>(row, skew, lo, hi, c, keep);
  } else {
    KeepNone keep;
    a = slice_triple<Ty, ENT, NT>(row, skew, lo, hi, c, keep);
  }
  if (tid == 0) part[blockIdx.x] = make_float4(a.m, a.s, a.w, 0.0f);
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
__device__ __forceinline__ int below(unsigned long long mask) {  // set bits of lower lanes
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

// The largest number of few low bits that at least k and at most k + slack of
// the N values per lane (of BITS bits) reach; the k-th largest itself where
// ties allow no such number.  Two bits a step, after a first one from the
// largest value's upper eight (a factor of four each): three steps of eight at
// usual rows.
template <int N, int BITS>
__device__ __forceinline__ uint32_t kth(const uint32_t* o, int k, int slack) {
  uint32_t top = o[0];
#pragma unroll
  for (int j = 1; j < N; ++j) top = max(top, o[j]);
  top = wave_max(top) >> (BITS - 8);
  bool guess = top >= 3;
  uint32_t r = guess ? (top - 3) << (BITS - 8) : 0;
  int bit = guess ? BITS - 8 : BITS - 2;
  while (bit >= 0) {
    const uint32_t t1 = r + (1u << bit), t2 = r + (2u << bit), t3 = r + (3u << bit);
    int n1 = 0, n2 = 0, n3 = 0;
    if constexpr (N == 8) {  // (three counts of up to 512 in one sum)
      uint32_t c1 = 0, c2 = 0, c3 = 0;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        c1 += o[j] >= t1 ? 1 : 0;
        c2 += o[j] >= t2 ? 1 : 0;
        c3 += o[j] >= t3 ? 1 : 0;
      }
      const uint32_t c = wave_sum(c1 | c2 << 10 | c3 << 20);
      n1 = (int)(c & 1023), n2 = (int)(c >> 10 & 1023), n3 = (int)(c >> 20);
    } else {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        n1 += __popcll(__ballot(o[j] >= t1));
        n2 += __popcll(__ballot(o[j] >= t2));
        n3 += __popcll(__ballot(o[j] >= t3));
      }
    }
    if (guess && n1 < k) {
      guess = false;
      r = 0;
      bit = BITS - 2;
      continue;
    }
    guess = false;
    r = n3 >= k ? t3 : n2 >= k ? t2 : n1 >= k ? t1 : r;
    const int n = n3 >= k ? n3 : n2 >= k ? n2 : n1;
    if (n >= k && n <= k + slack) break;
    bit -= 2;
  }
  return r;
}

// y[j], by halving (bits are chosen by a mask: a choice of elements by j would
// put y into memory)
template <int N>
__device__ __forceinline__ float element(const float (&y)[N], int j) {
  if constexpr (N == 1) {
    return y[0];
  } else {
    const uint32_t odd = 0u - (uint32_t)(j & 1);
    float h[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      h[i] = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, y[2 * i + 1]) & odd) |
                                           (__builtin_bit_cast(uint32_t, y[2 * i]) & ~odd));
    return element<N / 2>(h, j >> 1);
  }
}

// A candidate as one number: value first, then the lower column; no two of a
// row are equal.
__device__ __forceinline__ unsigned long long candidate(uint32_t order, int col) {
  return (unsigned long long)order << 32 | (uint32_t)~col;
}

// The k best of a whole row, whatever its ties: one wave reads it in order of
// columns, candidates wait in LDS, and a full list is cut to its k best, whose
// last one a later candidate must exceed (an equal value has a higher column).
// list: [QCAP], of which the first k are the result.  floor: an `ordered`
// number that at least k logits reach.
constexpr int QCAP = 1024;
__device__ int cut(unsigned long long* list, int n, int k, uint32_t& floor) {
  wave_lds();
  if (n <= k) return n;
  constexpr int N = QCAP / 64;
  const int lane = threadIdx.x & 63;
  unsigned long long e[N];
  uint32_t o[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    e[j] = j * 64 + lane < n ? list[j * 64 + lane] : 0ull;
    o[j] = (uint32_t)(e[j] >> 32);
  }
  const uint32_t last = kth<N, 32>(o, k, 0);
  int above = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) above += __popcll(__ballot(o[j] > last));
  int ties = k - above, m = 0;
  wave_lds();
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const bool tie = o[j] == last;  // (0 is no entry and below any)
    const unsigned long long eq = __ballot(tie);
    const bool keep = o[j] > last || (tie && below(eq) < ties);
    const unsigned long long mask = __ballot(keep);
    if (keep) list[m + below(mask)] = e[j];
    m += __popcll(mask);
    ties -= min(ties, (int)__popcll(eq));
  }
  floor = last + 1;
  wave_lds();
  return m;
}

template <class Ty>
__device__ void select_row(const typename Ty::E* row, int V, int k, uint32_t floor, unsigned long long* list) {
  constexpr int VE = Ty::VE;
  static_assert(64 * VE <= QCAP / 2, "a vector per lane fits behind a list that is not cut");
  const int lane = threadIdx.x & 63;
  int n = 0;
#pragma unroll 1
  for (int base = 0; base < V; base += 64 * VE) {
    float x[VE];
    const int i0 = base + lane * VE;
    if (i0 + VE <= V) {
      Ty::unpack(load16(row + i0), x);
    } else {
#pragma unroll
      for (int j = 0; j < VE; ++j) x[j] = i0 + j < V ? Ty::get(row[i0 + j]) : 0.0f;
    }
    int hit = 0, at = n, more = 0;
#pragma unroll
    for (int j = 0; j < VE; ++j) {
      const bool take = i0 + j < V && ordered(x[j]) >= floor;
      const unsigned long long mask = __ballot(take);
      hit |= take ? 1 << j : 0;
      at += below(mask);
      more += __popcll(mask);
    }
    if (more == 0) continue;
#pragma unroll
    for (int j = 0; j < VE; ++j)
      if (hit >> j & 1) list[at++] = candidate(ordered(x[j]), i0 + j);
    n += more;
    if (n > QCAP / 2) n = cut(list, n, k, floor);
  }
  cut(list, n, k, floor);
}

struct FinishArgs {
  int V, k, S, nb;
  long ld;
  float c, invtau;
};

// A row's outputs from its triple, by a workgroup of 256 threads.
//
// Top alternatives, the usual case: each thread holds up to HELD vectors of
// block maxima; a number that k of 128, 256 or 512 disjoint groups of them
// reach (4 groups and more for each alternative) leaves few more than k blocks
// and elements, and the place of each of those is the number of candidates
// above it.  Rows whose many candidates are no ties, or with more blocks than the
// registers hold, go through select_row.
//
// Latency bounds it, not bytes: the joining kernel takes 5.3 us for 1 and for 64
// rows of 151936 columns and 20 alternatives, a chain of dependent trips to
// memory (triples and maxima, then the chosen blocks) and the selection between.
// In cycles of one wave, with 20 / 128 alternatives: 2700 to the triple, 1700 to
// the groups, 1200 / 2600 the floor, 1100 / 1300 the blocks that reach it, 1200 /
// 5000 their elements, 3100 / 6500 the places.  (With lists that all waves
// filled through one counter: 4200 / 18600 for the elements, 6.4 us in all.)
constexpr int WAVE_BLOCKS = 128, WAVE_LIST = QCAP / 4, LISTED = 512;
constexpr int MAXKEYS = 4096;  // 262144 columns

// a row's given token: read at a kernel's start, since its two dependent loads
// would otherwise end the row's critical path
struct Given {
  int label;
  float x;
};
template <class Ty>
__device__ __forceinline__ Given given_of(const FinishArgs& f, const LogprobPtrs& q, int t) {
  Given g{-1, 0.0f};
  if (q.labels) g.label = q.labels[t];
  if (g.label >= 0 && g.label < f.V)
    g.x = Ty::get((static_cast<const typename Ty::E*>(q.logits) + (size_t)t * f.ld)[g.label]);
  return g;
}

// keys: the block maxima of the row, in LDS or memory; list: [QCAP] in LDS,
// which may be where the keys are
template <class Ty, bool TOP>
__device__ __forceinline__ void logprobs_finish(const FinishArgs& f, const LogprobPtrs& q, int t, const Given& g,
                                                const Triple& a, const u32x4* keys, unsigned long long* list) {
  typedef typename Ty::E E;
  typedef Blocks<Ty> B;
  constexpr int VE = Ty::VE, NT = 256, KV = 16 / sizeof(typename B::Key);
  constexpr int HELD = TOP ? MAXKEYS / KV / NT : 0;
  const int tid = threadIdx.x, lane = tid & 63;
  const E* row = static_cast<const E*>(q.logits) + (size_t)t * f.ld;
  const bool empty = a.s == 0.0f;
  const float l = log_sum(a, f.c);
  if (tid == NT - 1) {
    *reinterpret_cast<float2*>(q.stats + 2 * (size_t)t) = make_float2(a.m, l);
    if (q.entropy) q.entropy[t] = entropy_of(a);
    if (q.logp) {
      float lp = g.label == -1 ? 0.0f : NAN;
      if (g.label >= 0 && g.label < f.V) lp = empty ? -INFINITY : scaled(g.x, a.m, f.invtau) - l;
      q.logp[t] = lp;
    }
  }
  if constexpr (TOP) {
    __shared__ uint16_t cand[4][WAVE_BLOCKS];
    __shared__ uint32_t group[512];
    __shared__ int count[3][4], ties[4];
    constexpr int OVER = 1 << 24;
    // (waves interleaved by vectors: neighbouring columns are often good together)
    const int place = lane * 4 + (tid >> 6);
    u32x4 held[HELD];
    const int skew = skew_of<Ty>(row), end = f.V + skew;
    const int nvec = (end + B::TILE - 1) / B::TILE * B::PER_TILE / KV;
#pragma unroll
    for (int i = 0; i < HELD; ++i) held[i] = i * NT + place < nvec ? keys[i * NT + place] : u32x4{0, 0, 0, 0};
    // the best of each of eight groups per thread
    uint32_t best[8];
    if constexpr (KV == 8) {
      typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        uint32_t w0 = held[0][d];
        u16x2 m = __builtin_bit_cast(u16x2, w0);
#pragma unroll
        for (int i = 1; i < HELD; ++i) {
          const uint32_t w = held[i][d];
          m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w));
        }
        best[2 * d] = m[0];
        best[2 * d + 1] = m[1];
      }
    } else {
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        best[d] = held[0][d];
        best[4 + d] = held[1][d];
#pragma unroll
        for (int i = 2; i < HELD; i += 2) {
          best[d] = max(best[d], (uint32_t)held[i][d]);
          best[4 + d] = max(best[4 + d], (uint32_t)held[i + 1][d]);
        }
      }
    }
    // 512 groups in all, 8, 4 or 2 of a thread as fewer or more of them hold
    // vectors; each wave counts in all of them, to the same number
    const int shift = nvec <= 64 && KV == 8 ? 3 : nvec <= 128 ? 2 : 1;
    if (shift <= 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j) best[j] = max(best[j], best[4 + j]);
    }
    if (shift == 1) {
      best[0] = max(best[0], best[2]);
      best[1] = max(best[1], best[3]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < 1 << shift && place < 512 >> shift) group[(place << shift) + j] = best[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) best[j] = group[64 * j + lane];
    if (f.k <= 64) {
#pragma unroll
      for (int j = 0; j < 4; ++j) best[j] = max(best[j], best[4 + j]);
    }
    const int slack = f.k / 8 + 4;  // a few more candidates for fewer steps
    uint32_t floor;
    if (f.k > 64) {
      floor = kth<8, B::BITS>(best, f.k, slack);
    } else if (f.k > 24) {
      floor = kth<4, B::BITS>(best, f.k, slack);
    } else {
      best[0] = max(best[0], best[2]);
      best[1] = max(best[1], best[3]);
      floor = kth<2, B::BITS>(best, f.k, slack);
    }
    // (-inf and NaN rank alike, below any number, and each column reaches their
    // key: the floor where fewer than k groups or numbers above it are left)
    constexpr uint32_t LAST = 0x007FFFFFu >> (32 - B::BITS);
    floor = max(floor, LAST);
    // First the candidates that reach the floor.  If their blocks hold too many,
    // those that reach a higher one, from the blocks' vectors in 512 groups.
    // Then those above the floor: where ties did it (a masked or constant row)
    // they are few, and the lowest columns at the floor itself complete them.
    // Each wave reads the blocks it holds the maxima of, into a list of its own.
    const int wave = tid >> 6;
    unsigned long long* mine = list + wave * WAVE_LIST;
    int c[4];  // entries of the waves' lists
    bool done = false;
    int n = 0;
    uint32_t lo = floor;
    for (int step = 0; step < 3; ++step) {
      int nb = 0, nc = 0;
      uint32_t hits = 0;  // bit e: the e-th maximum held
      const uint32_t high = lo << (32 - B::BITS);
#pragma unroll
      for (int e = 0; e < HELD * KV; ++e) {
        const uint32_t w = held[e / KV][e % KV * 4 / KV];
        hits |= (KV == 8 && e % 2 == 0 ? w << 16 : w) >= high ? 1u << e : 0u;
      }
      for (unsigned long long mask; (mask = __ballot(hits != 0)) != 0; hits &= hits - 1) {
        const int at = nb + below(mask), e = __builtin_ctz(hits | 1u << 31);
        if (hits != 0 && at < WAVE_BLOCKS) cand[wave][at] = (uint16_t)((e / KV * NT + place) * KV + e % KV);
        nb += __popcll(mask);
      }
      wave_lds();
      const int nv = nb * B::VECS;
      // f(vector, position) for the blocks' vectors, 64 at a time; NaN where
      // there is no column
      const auto each = [&](auto&& f_) {
        constexpr int U = 4;  // vectors in flight per lane
        for (int base = 0; base < nv; base += 64 * U) {
          u32x4 x[U];
          int pos[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (base + 64 * u >= nv) break;
            const int at = base + 64 * u + lane;
            pos[u] = at < nv ? B::position(cand[wave][at / B::VECS], at % B::VECS) : end;
            x[u] = u32x4{~0u, ~0u, ~0u, ~0u};
            if (pos[u] >= skew && pos[u] + VE <= end) x[u] = load16(row + (pos[u] - skew));
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (base + 64 * u >= nv) break;
            float y[VE];
            Ty::unpack(x[u], y);
            if (__ballot(pos[u] < end && (pos[u] < skew || pos[u] + VE > end)) != 0) {
#pragma unroll
              for (int j = 0; j < VE; ++j) {
                const int col = pos[u] + j - skew;
                if (pos[u] < skew || pos[u] + VE > end) y[j] = col >= 0 && col < f.V ? Ty::get(row[col]) : NAN;
              }
            }
            f_(y, pos[u]);
          }
        }
      };
      // key(x) >= lo as a comparison of numbers, false for NaN; at the last key
      // every column takes part, NaN among them
      const bool all = lo == LAST;
      const float least = unordered(high);
      const bool over = nvec > HELD * NT || nb > WAVE_BLOCKS;
      if (!over) {
        each([&](const float (&y)[VE], int pos) {
          uint32_t in = 0;
          if (all) {
            in = (1u << max(min(end - pos, VE), 0)) - (1u << max(skew - pos, 0));
          } else {
#pragma unroll
            for (int j = 0; j < VE; ++j) in |= y[j] >= least ? 1u << j : 0u;
          }
          // (most lanes with any have one: the loop runs once or twice)
          for (unsigned long long mask; (mask = __ballot(in != 0)) != 0; in &= in - 1) {
            const int at = nc + below(mask), j = __builtin_ctz(in | 1u << 31);
            if (in != 0 && at < WAVE_LIST) mine[at] = candidate(ordered(element(y, j)), pos + j - skew);
            nc += __popcll(mask);
          }
        });
      }
      if (lane == 0) count[step][wave] = over ? OVER : nc;
      __syncthreads();
      n = 0;
      int most = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        c[w] = count[step][w];
        n += c[w];
        most = max(most, c[w]);
      }
      const bool fits = most <= WAVE_LIST && n <= LISTED;
      done = fits && (n >= f.k || lo > floor);
      if (done) break;
      if (step == 0 && !fits && most < OVER) {
        best[0] = best[1] = 0;
        each([&](const float (&y)[VE], int pos) {
          float top = y[0];
#pragma unroll
          for (int j = 1; j < VE; ++j) top = fmaxf(top, y[j]);
          const uint32_t key = pos < end ? B::key(top) : 0u;
          if (pos / VE & 1) best[1] = max(best[1], key);
          else best[0] = max(best[0], key);
        });
        group[tid] = best[0];
        group[NT + tid] = best[1];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) best[j] = group[64 * j + lane];
        floor = max(floor, kth<8, B::BITS>(best, f.k, slack));
        lo = floor;
      } else {
        lo = floor + 1;
      }
    }
    // at the floor itself, in order of columns, behind the last list
    unsigned long long* last = list + 3 * WAVE_LIST + c[3] - n;
    c[3] -= n;
    for (int base = 0; done && n < f.k && base < f.V; base += NT * VE) {
      const int c0 = base + tid * VE;
      int hit = 0, at = 0, total = 0;
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const bool in = c0 + j < f.V && B::key(Ty::get(row[c0 + j])) == floor;
        const unsigned long long mask = __ballot(in);
        hit |= in ? 1 << j : 0;
        at += below(mask);
        total += __popcll(mask);
      }
      if (lane == 0) ties[wave] = total;
      __syncthreads();
      total = 0;
      for (int w = 0; w < 4; ++w) {
        if (w == wave) at += total;
        total += ties[w];
      }
#pragma unroll
      for (int j = 0; j < VE; ++j)
        if (hit >> j & 1) {
          if (n + at < f.k) last[n + at] = candidate(ordered(Ty::get(row[c0 + j])), c0 + j);
          ++at;
        }
      n = min(f.k, n + total);
      __syncthreads();
    }
    c[3] += n;
    if (!done || n < f.k) {
      __syncthreads();
      if (tid < 64) select_row<Ty>(row, f.V, f.k, floor << (32 - B::BITS), list);
      c[0] = n = f.k;
      c[1] = c[2] = c[3] = 0;
    }
    // Places: each wave counts, for all candidates, those of its own list above
    // them.  The lists go up to multiples of eight (0 is below each candidate).
    uint32_t* places = group;
    places[tid] = places[NT + tid] = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      if (tid >> 3 == w && c[w] + (tid & 7) < ((c[w] + 7) & ~7)) list[w * WAVE_LIST + c[w] + (tid & 7)] = 0ull;
    __syncthreads();
    const auto entry = [&](int i) {
      const int w1 = c[0], w2 = w1 + c[1], w3 = w2 + c[2];
      return list[i < w1 ? i : i < w2 ? i - w1 + WAVE_LIST : i < w3 ? i - w2 + 2 * WAVE_LIST : i - w3 + 3 * WAVE_LIST];
    };
    const int own = wave == 0 ? c[0] : wave == 1 ? c[1] : wave == 2 ? c[2] : c[3];
    const auto count_above = [&](auto width) {
      constexpr int R = decltype(width)::value;  // candidates per lane
      for (int base = 0; base < n; base += 64 * R) {
        unsigned long long e[R];
        int above[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
          e[r] = base + 64 * r + lane < n ? entry(base + 64 * r + lane) : 0ull;
          above[r] = 0;
        }
        for (int j = 0; j < own; j += 8) {
#pragma unroll
          for (int h = 0; h < 8; h += 2) {
            const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(mine + j + h);
#pragma unroll
            for (int r = 0; r < R; ++r) above[r] += (o.x > e[r] ? 1 : 0) + (o.y > e[r] ? 1 : 0);
          }
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (base + 64 * r + lane < n && above[r] > 0) atomicAdd(&places[base + 64 * r + lane], above[r]);
      }
    };
    if (n <= 64) count_above(std::integral_constant<int, 1>{});
    else count_above(std::integral_constant<int, 3>{});
    __syncthreads();
    for (int i = tid; i < n; i += NT) {
      const int rank = (int)places[i];
      const unsigned long long e = entry(i);
      if (rank < f.k) {
        const float v = unordered((uint32_t)(e >> 32));
        const size_t at = (size_t)t * f.k + rank;
        q.top_idx[at] = (int)~(uint32_t)e;
        q.top_logp[at] = l != l ? NAN : empty ? -INFINITY : scaled(v, a.m, f.invtau) - l;
      }
    }
  }
}

template <class Ty, bool TOP>
__global__ __launch_bounds__(256, 4) void logprobs_finish_kernel(
    FinishArgs f, LogprobPtrs q, const float4* __restrict__ part,
    const typename Blocks<Ty>::Key* __restrict__ blocks) {
  const int t = blockIdx.x;
  const Given g = given_of<Ty>(f, q, t);
  const Triple a = row_triple(part + (size_t)t * f.S, f.S, f.c);
  if constexpr (TOP) {
    __shared__ __align__(16) unsigned long long list[QCAP];
    logprobs_finish<Ty, true>(f, q, t, g, a, reinterpret_cast<const u32x4*>(blocks + (size_t)t * f.nb), list);
  } else {
    logprobs_finish<Ty, false>(f, q, t, g, a, nullptr, nullptr);
  }
}

// A whole row by one workgroup, for rows enough to fill the chip: no triples
// and no block maxima through memory (writing 20 MB of them beside a read of
// 1.2 GB took 25 us).  (Six workgroups a CU of fp32 would spill a register.)
template <class Ty, bool ENT, bool TOP, bool NT>
__global__ __launch_bounds__(256, sizeof(typename Ty::E) == 2 ? 6 : 5) void logprobs_row_kernel(FinishArgs f,
                                                                                               LogprobPtrs q) {
  typedef typename Blocks<Ty>::Key Key;
  const int t = blockIdx.x;
  const typename Ty::E* row = static_cast<const typename Ty::E*>(q.logits) + (size_t)t * f.ld;
  const int skew = skew_of<Ty>(row);
  row -= skew;
  const Given g = given_of<Ty>(f, q, t);
  if constexpr (TOP) {
    __shared__ __align__(16) Key kept[MAXKEYS];
    static_assert(sizeof(kept) >= QCAP * 8, "the list of candidates takes the keys' place");
    KeepRow<Ty> keep{kept};
    const Triple a = slice_triple<Ty, ENT, NT>(row, skew, 0, f.V + skew, f.c, keep);
    logprobs_finish<Ty, true>(f, q, t, g, a, reinterpret_cast<const u32x4*>(kept),
                                 reinterpret_cast<unsigned long long*>(kept));
  } else {
    KeepNone keep;
    const Triple a = slice_triple<Ty, ENT, NT>(row, skew, 0, f.V + skew, f.c, keep);
    logprobs_finish<Ty, false>(f, q, t, g, a, nullptr, nullptr);
  }
}

// ------------------------------------------------------------------ teacher
// A row's teacher list over one wave: entry lane + 64 i in register i < TI (1 or
// 4: lists of up to 64 or 256).
// ix -1: an entry without weight.  bad: an entry is out of range, NaN or
// +inf; any: some entry has weight.
template <int TI>
struct Listed {  // as given: read ahead of what hides their way from memory
  int ix[TI];
  float v[TI];
  __device__ __forceinline__ Listed(const int* idx, const float* val, int k) {
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int at = (threadIdx.x & 63) + 64 * i;
      ix[i] = at < k ? idx[at] : -1;
      v[i] = at < k ? val[at] : -INFINITY;
    }
  }
};
template <int TI>
struct Teacher {
  int ix[TI];
  float q[TI], logq[TI];
  bool bad, any;

  __device__ __forceinline__ Teacher(const Listed<TI>& given, int V, float invtau) {
    float v[TI], mx = -INFINITY;
    bool b = false;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      ix[i] = given.ix[i];
      v[i] = ix[i] == -1 ? -INFINITY : given.v[i];
      b |= ix[i] < -1 || ix[i] >= V || v[i] != v[i] || v[i] == INFINITY;
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

struct DistillPtrs {
  const void* logits;
  const int* idx;
  const float* teacher;
  float* loss;
  float* stats;
};

// by one wave
template <class Ty, int TI>
__device__ __forceinline__ void distill_finish(const FinishArgs& f, const DistillPtrs& q, int t, const Teacher<TI>& te,
                                               const float (&x)[TI], const Triple& a) {
  const float l = log_sum(a, f.c);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < TI; ++i)
    if (te.ix[i] >= 0) {
      // q (log q - log p), the far end of log p kept in range by its q (a
      // listed column may be masked at the type's lowest value; at -inf, as in
      // an empty row, it is infinite however small q / tau)
      const float far = scaled(x[i], a.m, te.q[i] * f.invtau);
      sum += x[i] == -INFINITY && l == l ? INFINITY : fmaf(te.q[i], te.logq[i] + l, -far);
    }
  sum = wave_sum(sum);
  if (threadIdx.x == 0) {
    q.loss[t] = te.bad ? NAN : sum;
    *reinterpret_cast<float2*>(q.stats + 2 * (size_t)t) = make_float2(a.m, l);
  }
}

template <int TI>
__device__ __forceinline__ Listed<TI> listed_row(const FinishArgs& f, const DistillPtrs& q, int t) {
  return Listed<TI>(q.idx + (size_t)t * f.k, q.teacher + (size_t)t * f.k, f.k);
}
template <class Ty, int TI>
__device__ __forceinline__ Teacher<TI> teacher_row(const FinishArgs& f, const DistillPtrs& q, int t,
                                                   const Listed<TI>& given, float (&x)[TI]) {
  const typename Ty::E* row = static_cast<const typename Ty::E*>(q.logits) + (size_t)t * f.ld;
  const Teacher<TI> te(given, f.V, f.invtau);
#pragma unroll
  for (int i = 0; i < TI; ++i) x[i] = te.ix[i] >= 0 ? Ty::get(row[te.ix[i]]) : 0.0f;
  return te;
}

template <class Ty, int TI>
__global__ __launch_bounds__(64) void distill_finish_kernel(FinishArgs f, DistillPtrs q,
                                                            const float4* __restrict__ part) {
  const int t = blockIdx.x;
  float x[TI];
  const Teacher<TI> te = teacher_row<Ty, TI>(f, q, t, listed_row<TI>(f, q, t), x);
  distill_finish<Ty, TI>(f, q, t, te, x, row_triple(part + (size_t)t * f.S, f.S, f.c));
}

template <class Ty, int TI, bool NT>
__global__ __launch_bounds__(256) void distill_row_kernel(FinishArgs f, DistillPtrs q) {
  const int t = blockIdx.x;
  const typename Ty::E* row = static_cast<const typename Ty::E*>(q.logits) + (size_t)t * f.ld;
  const int skew = skew_of<Ty>(row);
  const Listed<TI> given = listed_row<TI>(f, q, t);
  KeepNone keep;
  const Triple a = slice_triple<Ty, false, NT>(row - skew, skew, 0, f.V + skew, f.c, keep);
  if (threadIdx.x >= 64) return;
  float x[TI];
  const Teacher<TI> te = teacher_row<Ty, TI>(f, q, t, given, x);
  distill_finish<Ty, TI>(f, q, t, te, x, a);
}

// ----------------------------------------------------------------- backward
// d_logits = p fma(max(log2 p, clamp), ga, gb) (+ gl / tau at the label) with
// log2 p = c (x - m) - l log2 e:
//   logprobs  ga = -g_H ln 2 / tau, gb = -(g_logp + g_H H) / tau
//   distill   ga = 0, gb = g / tau (the listed columns follow)
//
// A workgroup has one tile of a row, BU vectors a thread: loaded at once,
// computed, stored.  Time goes by the bytes (4096 x 151936 bf16, read and
// written, us): 477 with two slices a row, cached, 449 with a tile a workgroup,
// 401 of 4 vectors streamed, 381 of 2, 408 of 1.  The distillation's
// workgroups also read the teacher's list, which 4 vectors repay better (198 us
// at half the rows; 210 of 2).
constexpr int BU_LOGPROBS = 2, BU_DISTILL = 4;

template <class Ty, int BU>
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

// A workgroup's tile of a row: positions [lo, hi), from `skew` on where lo is
// 0; row, out: where position 0 would be.
template <class Ty, int BU, bool ACC, bool NT>
struct Tile {
  typedef typename Ty::E E;
  static constexpr int VE = Ty::VE, SIZE = bwd_tile<Ty, BU>();
  const E* row;
  E* out;
  int skew, lo, hi;
  u32x4 v[BU], old[ACC ? BU : 1];

  __device__ __forceinline__ Tile(const E* r, E* o, int sk, int l, int V)
      : row(r - sk), out(o - sk), skew(sk), lo(l), hi(min(V + sk, l + SIZE)) {}
  __device__ __forceinline__ int first(int u) const { return lo + (u * 256 + (int)threadIdx.x) * VE; }
  __device__ __forceinline__ bool whole(int i0) const { return i0 >= skew && i0 + VE <= hi; }

  // no partial vector in the tile: known to all its threads alike, so that the
  // loads stand in no branch of their own
  __device__ __forceinline__ bool full() const { return lo >= skew && lo + SIZE <= hi; }

  __device__ __forceinline__ void load() {
    if (!full()) return;
#pragma unroll
    for (int u = 0; u < BU; ++u) {
      v[u] = stream16<NT>(row + first(u));
      if constexpr (ACC) old[u] = stream16<NT>(out + first(u));
    }
  }

  // grad(x, i0): the gradient of the vector at position i0 in place of x
  template <class F>
  __device__ __forceinline__ void store(F grad) {
    if (full()) {
#pragma unroll
      for (int u = 0; u < BU; ++u) {
        float x[VE], o[VE];
        Ty::unpack(v[u], x);
        if constexpr (ACC) Ty::unpack(old[u], o);
        grad(x, first(u));
#pragma unroll
        for (int j = 0; j < VE; ++j) x[j] += ACC ? o[j] : 0.0f;
        stream16<NT>(out + first(u), Ty::pack(x));
      }
      return;
    }
#pragma unroll 1
    for (int u = 0; u < BU; ++u) {
      const int i0 = first(u);
      float x[VE], o[VE];
      if (whole(i0)) {
        Ty::unpack(stream16<NT>(row + i0), x);
        if constexpr (ACC) Ty::unpack(stream16<NT>(out + i0), o);
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          const bool in = i0 + j >= skew && i0 + j < hi;
          x[j] = in ? Ty::get(row[i0 + j]) : 0.0f;
          o[j] = ACC && in ? Ty::get(out[i0 + j]) : 0.0f;
        }
      }
      grad(x, i0);
#pragma unroll
      for (int j = 0; j < VE; ++j) x[j] += ACC ? o[j] : 0.0f;
      if (whole(i0)) {
        stream16<NT>(out + i0, Ty::pack(x));
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (i0 + j >= skew && i0 + j < hi) out[i0 + j] = Ty::put(x[j]);
      }
    }
  }

  // the same value everywhere (zeros add nothing)
  __device__ __forceinline__ void fill(float value) {
    if (ACC && value == 0.0f) return;
    float x[VE];
#pragma unroll
    for (int j = 0; j < VE; ++j) x[j] = value;
#pragma unroll 1
    for (int u = 0; u < BU; ++u) {
      const int i0 = first(u);
      if (whole(i0)) {
        stream16<NT>(out + i0, Ty::pack(x));
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (i0 + j >= skew && i0 + j < hi) out[i0 + j] = Ty::put(value);
      }
    }
  }
};

enum { ZEROS = 1, NANS = 2 };  // a row of one value

// row and tile of a workgroup, in scalar registers
struct Place {
  int t, tile;
  __device__ __forceinline__ explicit Place(int S)
      : t(__builtin_amdgcn_readfirstlane((int)(blockIdx.x / (unsigned)S))), tile((int)blockIdx.x - t * S) {}
};

struct BwdArgs {
  int V, k, S;
  long ld, ldg;
  float c, invtau;
};

template <class Ty, bool ACC, bool NT>
__global__ __launch_bounds__(256) void logprobs_bwd_kernel(BwdArgs b, LogprobGradPtrs q) {
  typedef typename Ty::E E;
  typedef Tile<Ty, BU_LOGPROBS, ACC, NT> Part;
  const Place at_tile(b.S);
  const int t = at_tile.t;
  const E* row = static_cast<const E*>(q.logits) + (size_t)t * b.ld;
  const int skew = skew_of<Ty>(row);
  Part part(row, static_cast<E*>(q.d_logits) + (size_t)t * b.ldg, skew, at_tile.tile * Part::SIZE, b.V);
  const float2 st = *reinterpret_cast<const float2*>(q.stats + 2 * (size_t)t);
  // (each load on its own: none waits for another's value)
  const int lab = q.labels ? q.labels[t] : -1;
  const float given = q.g_logp ? q.g_logp[t] : 0.0f, gl = lab == -1 ? 0.0f : given;
  const float ge = q.g_entropy ? q.g_entropy[t] : 0.0f, ent = q.g_entropy ? q.entropy[t] : 0.0f;
  const int same = gl == 0.0f && ge == 0.0f ? ZEROS : lab < -1 || lab >= b.V ? NANS : st.y == -INFINITY ? ZEROS : 0;
  if (same != 0) return part.fill(same == ZEROS ? 0.0f : NAN);
  part.load();
  const float H = ge != 0.0f ? ent : 0.0f;
  const RowGrad g{st.x, b.c, st.y * LOG2E, -ge * LN2 * b.invtau, -fmaf(ge, H, gl) * b.invtau};
  const float at = gl * b.invtau;
  part.store([&](float (&x)[Ty::VE], int i0) {
#pragma unroll
    for (int j = 0; j < Ty::VE; ++j) x[j] = g(x[j]);
    const int here = lab + skew - i0;
    if ((unsigned)here < (unsigned)Ty::VE) {
#pragma unroll
      for (int j = 0; j < Ty::VE; ++j) x[j] += here == j ? at : 0.0f;
    }
  });
}

template <class Ty, int TI, bool ACC, bool NT>
__global__ __launch_bounds__(256) void distill_bwd_kernel(BwdArgs b, const typename Ty::E* logits,
                                                          const int* __restrict__ idx,
                                                          const float* __restrict__ teacher,
                                                          const float* __restrict__ stats,
                                                          const float* __restrict__ g_loss, typename Ty::E* d_logits) {
  typedef typename Ty::E E;
  typedef Tile<Ty, BU_DISTILL, ACC, NT> Part;
  __shared__ __align__(16) int lidx[64 * TI + 4];
  __shared__ __align__(16) float lq[64 * TI + 4];
  const Place at_tile(b.S);
  const int t = at_tile.t, tid = threadIdx.x;
  const E* row = logits + (size_t)t * b.ld;
  E* out = d_logits + (size_t)t * b.ldg;
  const int skew = skew_of<Ty>(row);
  Part part(row, out, skew, at_tile.tile * Part::SIZE, b.V);
  const float g = g_loss[t];
  const float2 st = *reinterpret_cast<const float2*>(stats + 2 * (size_t)t);
  // (each wave computes the list; all get the same)
  const Teacher<TI> te(Listed<TI>(idx + (size_t)t * b.k, teacher + (size_t)t * b.k, b.k), b.V, b.invtau);
  const int same = g == 0.0f ? ZEROS : te.bad ? NANS : !te.any || st.y == -INFINITY ? ZEROS : 0;
  if (same != 0) return part.fill(same == ZEROS ? 0.0f : NAN);
  const RowGrad r{st.x, b.c, st.y * LOG2E, 0.0f, g * b.invtau};
  // the entries of this tile, in list order
  int n = 0;
#pragma unroll
  for (int i = 0; i < TI; ++i) {
    const bool in = te.ix[i] >= 0 && te.ix[i] + skew >= part.lo && te.ix[i] + skew < part.hi;
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
  const int mine = tid < n ? lidx[tid] : 0;
  float v = 0.0f;
  if (tid < n) {
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
  part.load();  // (ahead of a barrier they would only be waited for there)
  part.store([&](float (&x)[Ty::VE], int) {
#pragma unroll
    for (int j = 0; j < Ty::VE; ++j) x[j] = exp2_hw(r.log2p(x[j])) * r.gb;
  });
  __syncthreads();  // the tile's own writes come before the listed columns'
  if (tid < n) out[mine] = Ty::put(v);
}

// --------------------------------------------------------------- host side
// positions of a row at most
template <class Ty>
int positions(const VocabDims& d) {
  return d.V + (sizeof(typename Ty::E) == 2 ? 1 : 0);
}

// Slices of a row: `want` workgroups, at least a tile each.
struct Split {
  int S, slice;
};
Split split(int T, int V, int tile, long want) {
  const long tiles = ((long)V + tile - 1) / tile;
  const long S = std::min((want + T - 1) / T, tiles);
  const long per = (tiles + S - 1) / S;
  return Split{(int)((tiles + per - 1) / per), (int)(per * tile)};
}
constexpr long WANT = 4096;
template <class Ty>
int blocks_of(const VocabDims& d) {
  return (positions<Ty>(d) + fwd_tile<Ty>() - 1) / fwd_tile<Ty>() * Blocks<Ty>::PER_TILE;
}
// A workgroup per row, with its block maxima in LDS where they are wanted:
// from MANY_ROWS on, and for short rows, where one launch costs less than a
// row's slices gain.  Measured (us, whole row / slices, the time of a call,
// which two launches hold at 13 or more; on the GPU alone the slices of few
// rows take 8.5 and with alternatives 10; the limits are the same for both
// types and for calls with and without entropy): bf16 of 151936 columns with 20
// alternatives 1 row 18.9 / 14.9, 64 rows 20.7 / 15.8, 200 rows 23.2 / 23.4,
// 400 rows 30.4 / 32.9, 4096 rows 202 / 234; without 64 rows 16.2 / 13.7, 200
// rows 20.1 / 17.7, 400 rows 26.3 / 27.8; of 32003 columns with 20
// alternatives 1 row 10.5 / 14.6, 400 rows 18.4 / 20.8; fp32 of 50021 columns
// without 1 row 9.0 / 13.3, 57 rows 9.5 / 14.2, with 20 alternatives 12.3 /
// 14.7 and 13.5 / 14.8.  So the other side is the faster one for 200 to
// somewhat less than 400 rows of 151936 columns without alternatives (2.4 us at
// 200) and for fp32 rows of 50021 columns with them (2.4 us for 1 row, 1.3 for
// 57).
constexpr int MANY_ROWS = 200, SHORT = 65536, SHORT_TOP = 32768;
template <class Ty>
bool whole_rows(const VocabDims& d, bool top) {
  if (top && blocks_of<Ty>(d) > MAXKEYS) return false;
  return d.T >= MANY_ROWS || d.V <= (top ? SHORT_TOP : SHORT);
}
template <class Ty>
Split fwd_split(const VocabDims& d) {
  return split(d.T, positions<Ty>(d), fwd_tile<Ty>(), WANT);
}
template <class Ty>
size_t part_bytes(const VocabDims& d) {
  return (size_t)d.T * fwd_split<Ty>(d).S * sizeof(float4);
}
template <class Ty>
FinishArgs finish_args(const VocabDims& d, int S) {
  return FinishArgs{d.V, d.k, S, blocks_of<Ty>(d), d.ld, d.invtau * LOG2E, d.invtau};
}
// Logits of more bytes than this (and their gradients) are streamed past the
// caches; 256 MB of them in front of the memory keep fewer for whoever comes
// next.  Measured, bf16, 151936 columns, us kept / streamed, logits just
// written by another kernel: 256 rows (78 MB) distillation 16.5 / 21.3, policy
// gradient 23.3 / 23.5; 512 rows (156 MB) 23.0 / 25.8 and 48.3 / 38.4; 1024
// rows (311 MB) 63.2 / 52.7 and 100.3 / 80.2.
constexpr long STREAM_BYTES = 128L << 20;
bool streamed(const VocabDims& d) { return (long)d.T * d.V * (d.f32 ? 4 : 2) > STREAM_BYTES; }
// f(true_type) or f(false_type)
template <class F>
void choose(bool b, F&& f) {
  b ? f(std::true_type{}) : f(std::false_type{});
}

template <class Ty, int BU>
BwdArgs bwd_args(const VocabDims& d) {
  const int tile = bwd_tile<Ty, BU>();
  return BwdArgs{d.V, d.k, (positions<Ty>(d) + tile - 1) / tile, d.ld, d.ldg, d.invtau * LOG2E, d.invtau};
}

template <class Ty, bool ENT, bool TOP, bool NT>
void stats_launch(const VocabDims& d, const Split& s, const void* logits, char* ws, hipStream_t st) {
  typedef typename Ty::E E;
  hipLaunchKernelGGL((vocab_stats_kernel<Ty, ENT, TOP, NT>), dim3((size_t)d.T * s.S), dim3(256), 0, st,
                     static_cast<const E*>(logits), d.ld, d.V, s.S, s.slice, d.invtau * LOG2E,
                     reinterpret_cast<float4*>(ws),
                     reinterpret_cast<typename Blocks<Ty>::Key*>(ws + part_bytes<Ty>(d)), blocks_of<Ty>(d));
}

template <class Ty, bool ENT, bool TOP, bool NT>
void logprobs_launch(const VocabDims& d, const LogprobPtrs& q, char* ws, hipStream_t st) {
  if (whole_rows<Ty>(d, TOP)) {
    hipLaunchKernelGGL((logprobs_row_kernel<Ty, ENT, TOP, NT>), dim3(d.T), dim3(256), 0, st, finish_args<Ty>(d, 1),
                       q);
    return;
  }
  const Split s = fwd_split<Ty>(d);
  const float4* part = reinterpret_cast<const float4*>(ws);
  const auto* blocks = reinterpret_cast<const typename Blocks<Ty>::Key*>(ws + part_bytes<Ty>(d));
  const FinishArgs f = finish_args<Ty>(d, s.S);
  stats_launch<Ty, ENT, TOP, NT>(d, s, q.logits, ws, st);
  hipLaunchKernelGGL((logprobs_finish_kernel<Ty, TOP>), dim3(d.T), dim3(256), 0, st, f, q, part, blocks);
}

template <class Ty>
void logprobs_launch(const VocabDims& d, const LogprobPtrs& q, char* ws, hipStream_t st) {
  choose(q.entropy != nullptr, [&](auto ent) {
    choose(d.k > 0, [&](auto top) {
      choose(streamed(d), [&](auto nt) {
        logprobs_launch<Ty, decltype(ent)::value, decltype(top)::value, decltype(nt)::value>(d, q, ws, st);
      });
    });
  });
}

template <class Ty, int TI, bool NT>
void distill_launch(const VocabDims& d, const DistillPtrs& q, char* ws, hipStream_t st) {
  if (whole_rows<Ty>(d, false)) {
    hipLaunchKernelGGL((distill_row_kernel<Ty, TI, NT>), dim3(d.T), dim3(256), 0, st, finish_args<Ty>(d, 1), q);
    return;
  }
  const Split s = fwd_split<Ty>(d);
  stats_launch<Ty, false, false, NT>(d, s, q.logits, ws, st);
  hipLaunchKernelGGL((distill_finish_kernel<Ty, TI>), dim3(d.T), dim3(64), 0, st, finish_args<Ty>(d, s.S), q,
                     reinterpret_cast<const float4*>(ws));
}

template <class Ty>
void logprobs_bwd_launch(const VocabDims& d, const LogprobGradPtrs& q, hipStream_t st) {
  const BwdArgs b = bwd_args<Ty, BU_LOGPROBS>(d);
  choose(d.accumulate, [&](auto acc) {
    choose(streamed(d), [&](auto nt) {
      hipLaunchKernelGGL((logprobs_bwd_kernel<Ty, decltype(acc)::value, decltype(nt)::value>),
                         dim3((size_t)d.T * b.S), dim3(256), 0, st, b, q);
    });
  });
}

template <class Ty, int TI>
void distill_bwd_launch(const VocabDims& d, const void* logits, const int* idx, const float* teacher,
                        const float* stats, const float* g_loss, void* d_logits, hipStream_t st) {
  typedef typename Ty::E E;
  const BwdArgs b = bwd_args<Ty, BU_DISTILL>(d);
  choose(d.accumulate, [&](auto acc) {
    choose(streamed(d), [&](auto nt) {
      hipLaunchKernelGGL((distill_bwd_kernel<Ty, TI, decltype(acc)::value, decltype(nt)::value>),
                         dim3((size_t)d.T * b.S), dim3(256), 0, st, b, static_cast<const E*>(logits), idx, teacher,
                         stats, g_loss, static_cast<E*>(d_logits));
    });
  });
}

// f(type, entries of a teacher list per lane)
template <class F>
void teacher_shape(const VocabDims& d, F&& f) {
  using One = std::integral_constant<int, 1>;
  using Four = std::integral_constant<int, 4>;
  if (d.f32) d.k <= 64 ? f(F32{}, One{}) : f(F32{}, Four{});
  else d.k <= 64 ? f(Bf16{}, One{}) : f(Bf16{}, Four{});
}

}  // namespace

template <class Ty>
static size_t ws_bytes_of(const VocabDims& d) {
  if (whole_rows<Ty>(d, d.k > 0)) return 0;  // (then a distillation's rows are whole too)
  return part_bytes<Ty>(d) + (d.k > 0 ? (size_t)d.T * blocks_of<Ty>(d) * sizeof(typename Blocks<Ty>::Key) : 0);
}
size_t vocab_ws_bytes(const VocabDims& d) { return d.f32 ? ws_bytes_of<F32>(d) : ws_bytes_of<Bf16>(d); }

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
  const DistillPtrs q{logits, idx, teacher, loss, stats};
  teacher_shape(d, [&](auto ty, auto ti) {
    choose(streamed(d), [&](auto nt) {
      distill_launch<decltype(ty), decltype(ti)::value, decltype(nt)::value>(d, q, ws, st);
    });
  });
  return hipGetLastError();
}

hipError_t launch_distill_bwd(const VocabDims& d, const void* logits, const int* idx, const float* teacher,
                              const float* stats, const float* g_loss, void* d_logits, hipStream_t st) {
  ProfScope prof(st, "vocab.distill_bwd");
  teacher_shape(d, [&](auto ty, auto ti) {
    distill_bwd_launch<decltype(ty), decltype(ti)::value>(d, logits, idx, teacher, stats, g_loss, d_logits, st);
  });
  return hipGetLastError();
}

}  // namespace oft
