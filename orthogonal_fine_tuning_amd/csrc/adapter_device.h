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

// The partial slots of an adapter of `pieces` pieces, from `first` on, clipped
// to those there are.
__device__ __forceinline__ int slots_of(const RowLists& l, const int* tiles, int list, int ad, int pieces, int& first) {
  const int all = RowLists::slots(list);
  first = min(max(tiles[l.part_at(list) + ad], 0), all);
  return min(pieces, all - first);
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

// 16-byte loads and stores; STREAM: past the caches, for rows that are read
// and written once and do not fit them.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
template <bool STREAM>
__device__ __forceinline__ uint4 load16(const void* p) {
  if constexpr (STREAM) return __builtin_bit_cast(uint4, __builtin_nontemporal_load(static_cast<const u32x4*>(p)));
  else return *static_cast<const uint4*>(p);
}
template <bool STREAM>
__device__ __forceinline__ void store16(void* p, const uint4& v) {
  if constexpr (STREAM) __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), static_cast<u32x4*>(p));
  else *static_cast<uint4*>(p) = v;
}

// Eight consecutive elements of a bf16 or fp32 row as P operands (P = 1 for
// bf16, whose values are operands already; 3 for fp32).
template <bool F32>
struct Oct;
template <>
struct Oct<false> {
  static constexpr int P = 1;
  uint4 u;
  template <bool STREAM = false>
  __device__ __forceinline__ void load(const void* p, size_t at) {
    u = load16<STREAM>(static_cast<const uint16_t*>(p) + at);
  }
  template <bool STREAM = false>
  __device__ __forceinline__ void store(void* p, size_t at) const {
    store16<STREAM>(static_cast<uint16_t*>(p) + at, u);
  }
  __device__ __forceinline__ void zero() { u = zero4(); }
  __device__ __forceinline__ void parts(uint4 (&o)[1]) const { o[0] = u; }
};
template <>
struct Oct<true> {
  static constexpr int P = 3;
  float4 a, b;
  template <bool STREAM = false>
  __device__ __forceinline__ void load(const void* p, size_t at) {
    const float* q = static_cast<const float*>(p) + at;
    a = __builtin_bit_cast(float4, load16<STREAM>(q));
    b = __builtin_bit_cast(float4, load16<STREAM>(q + 4));
  }
  template <bool STREAM = false>
  __device__ __forceinline__ void store(void* p, size_t at) const {
    float* q = static_cast<float*>(p) + at;
    store16<STREAM>(q, __builtin_bit_cast(uint4, a));
    store16<STREAM>(q + 4, __builtin_bit_cast(uint4, b));
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void parts(uint4 (&o)[3]) const {
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    split_bf16x8<3>(v, o);
  }
};

// A wave's own tile in LDS, 64 rows of 128 bytes, between the two ways in
// which its lanes hold it: by rows (piece i: 16 bytes of row 8 i + lane / 8,
// eight lanes to a row, as global memory is best read and written: a load
// whose lanes follow each other down the rows takes the memory pipe four
// times as long) and by operands (16 bytes of row 16 i + lane % 16, as matrix
// steps take and leave them).  Chunks of a row are exchanged by bits of its
// number, so that both ways touch all banks evenly.
struct WaveTile {
  static constexpr int BYTES = 64 * 128;
  char* lds;
  __device__ __forceinline__ uint4* at(int row, int chunk) const {
    return reinterpret_cast<uint4*>(lds + row * 128 + 16 * (chunk ^ ((row >> 1) & 7)));
  }
  __device__ __forceinline__ uint4& by_row(int i, int lane) const { return *at(8 * i + (lane >> 3), lane & 7); }
  __device__ __forceinline__ uint4& by_operand(int i, int chunk, int lane) const {
    return *at(16 * i + (lane & 15), chunk);
  }
};
// Between the accesses of different lanes to the wave's tile: LDS takes them
// in order, the compiler must not exchange them.
__device__ __forceinline__ void wave_order() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// The rows of a 64-row entry for the pieces of a tile (the last row again
// past the end)
__device__ __forceinline__ void tile_rows8(const RowLists& l, const int* order, const int4& e, int lane, int (&row)[8]) {
  const int mine = row_at(l, order, e.y + min(lane, e.z - 1));
#pragma unroll
  for (int i = 0; i < 8; ++i) row[i] = __shfl(mine, 8 * i + (lane >> 3));
}

// The rows of a piece, IDX at a time, in LDS: numbers fetched along with the
// rows themselves would wait for them (loads come back in order), and a fetch
// two steps ahead would be none.  IDX rows are also what one accumulator sums
// up before that goes onto the sum of those before it: a piece may have a
// million rows, and each of the last matrix steps of one long chain would be
// rounded to the whole sum's step.  (Sums of 65536 rows of two adapters beside
// QKV 297 us in one chain, 316 in chains of IDX rows, the rotation's 524 with
// either; pieces of fewer rows take as long as they did.)
constexpr int IDX = 2048;
__device__ __forceinline__ void fetch_rows(const RowLists& l, const int* order, int pos, int rows, int* idx) {
  for (int i = threadIdx.x; i < rows; i += blockDim.x) idx[i] = row_at(l, order, pos + i);
}

// Rows of more bytes than this are streamed past the caches: two batches in
// turn and one again and again, rotated in us, streamed and not: 76 MB 36, 38
// and 36, 30; 129 MB 55, 60 and 56, 52; 222 MB 92, 98 and 92, 99; low-rank
// updates of 129 MB 66, 74 and 67, 73, of 76 MB 44, 49 and 44, 40.  Where the
// two differ, rows are taken to be in the caches: the projection has just
// written them.
constexpr size_t STREAM_BYTES = (size_t)128 << 20;

}  // namespace oft
