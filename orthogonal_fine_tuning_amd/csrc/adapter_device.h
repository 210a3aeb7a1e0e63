// Device helpers of the kernels on adapters of many requests.
#pragma once

#include "oft_adapter.h"
#include "oft_device.h"

namespace oft {

__device__ __forceinline__ f32x4 mfma16(const bf16x8& a, const bf16x8& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Entry i of a list, false past its end (a grid is sized for the longest
// list that T rows can make).  An entry is clipped to the rows and adapters
// there are.
__device__ __forceinline__ bool list_entry(const RowLists& l, const int* tiles, int list, int i, int4& e) {
  if (i >= min(tiles[list], l.cap(list))) return false;
  e = *reinterpret_cast<const int4*>(tiles + l.list_at(list) + 4 * (size_t)i);
  e.x = e.x < l.n ? e.x : -1;
  e.y = min(max(e.y, 0), l.T - 1);
  e.z = min(min(e.z, l.rows_of(list)), l.T - e.y);
  return e.z > 0;
}

// the row at position `pos` of the order
__device__ __forceinline__ int row_at(const RowLists& l, const int* order, int pos) {
  return min(max(order[pos], 0), l.T - 1);
}

// fp32 in P parts of bf16, largest first, whose sum is the value: each part
// takes the next eight significant bits by truncation (rounding could carry
// the largest values to infinity), so that three parts hold all 24 bits and
// two parts 16.  Infinities and NaN stay whole in the first part.
template <int P>
__device__ __forceinline__ void split_bf16(float v, uint32_t (&h)[P]) {
  uint32_t u = __builtin_bit_cast(uint32_t, v);
  const bool finite = (u & 0x7F800000u) != 0x7F800000u;
  u |= (v != v) ? 0x400000u : 0u;  // a NaN whose set bits all lie below the first part
  h[0] = u >> 16;
#pragma unroll
  for (int p = 1; p < P; ++p) {
    v = v - __builtin_bit_cast(float, (uint32_t)h[p - 1] << 16);
    h[p] = finite ? __builtin_bit_cast(uint32_t, v) >> 16 : 0u;
  }
}

// eight fp32 -> P matrix-core operands
template <int P>
__device__ __forceinline__ void split_bf16x8(const float (&v)[8], uint4 (&o)[P]) {
  uint32_t w[P][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t a[P], b[P];
    split_bf16<P>(v[2 * i], a);
    split_bf16<P>(v[2 * i + 1], b);
#pragma unroll
    for (int p = 0; p < P; ++p) w[p][i] = a[p] | (b[p] << 16);
  }
#pragma unroll
  for (int p = 0; p < P; ++p) o[p] = make_uint4(w[p][0], w[p][1], w[p][2], w[p][3]);
}

// Eight consecutive elements of a bf16 or fp32 row as P operands (P = 1 for
// bf16, whose values are operands already; 3 for fp32).
template <bool F32>
struct Oct;
template <>
struct Oct<false> {
  static constexpr int P = 1;
  uint4 u;
  __device__ __forceinline__ void load(const void* p, size_t at) {
    u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
  }
  __device__ __forceinline__ void zero() { u = zero4(); }
  __device__ __forceinline__ void parts(uint4 (&o)[1]) const { o[0] = u; }
};
template <>
struct Oct<true> {
  static constexpr int P = 3;
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, size_t at) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    a = q[0];
    b = q[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void parts(uint4 (&o)[3]) const {
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    split_bf16x8<3>(v, o);
  }
};

}  // namespace oft
