// Internal interface of the kernels on adapters of many requests (host side
// and the device view of the rows' order).  The C-ABI layer (adapter_abi.cpp)
// validates every argument before calling these.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace oft {

constexpr int MAX_ADAPTERS = 1024;
constexpr int MAX_SEG = 8;

// Work lists over the rows in adapter order, in the caller's `tiles` buffer.
// An entry is {adapter, first position in `order`, rows, partial slot}; rows
// without an adapter come last, as entries of adapter -1.
//   LIST_16     16-row tiles, built for T <= T16_MAX only
//   LIST_64     64-row tiles
//   LIST_LONG   pieces of an adapter's rows for sums over rows, about a
//   LIST_SHORT  quarter (sixteenth) of all rows each.  An adapter of two or
//               more pieces gets a partial slot for each (`part` counts them
//               up to the adapter); one of a single piece has slot -1.
enum : int { LIST_16 = 0, LIST_64 = 1, LIST_LONG = 2, LIST_SHORT = 3, LISTS = 4 };
constexpr int T16_MAX = 2048;

struct RowLists {
  int T, n;
  // tiles and pieces of one adapter, and their rows
  __host__ __device__ int rows_of(int list) const {
    const int div = list == LIST_LONG ? 4 : 16;
    const int piece = ((T + div - 1) / div + 63) & ~63;
    return list == LIST_16 ? 16 : list == LIST_64 || piece < 64 ? 64 : piece;
  }
  __host__ __device__ int count(int list, int rows) const {
    if (list == LIST_16 && T > T16_MAX) return 0;
    const int c = rows_of(list);
    return (rows + c - 1) / c;
  }
  // entries at most: each of the n + 1 groups has one that is not full
  __host__ __device__ int cap(int list) const {
    if (list == LIST_16 && T > T16_MAX) return 0;
    const int c = T / rows_of(list) + n + 1;
    return c < T ? c : T;
  }
  // partial slots at most: a piece's adapter holds more than one piece's rows
  static __host__ __device__ int slots(int list) { return list == LIST_LONG ? 8 : 32; }
  // buffer, in int32: counts, the adapters' first partial slots, the lists
  __host__ __device__ size_t part_at(int list) const { return 8 + (list == LIST_SHORT ? (size_t)((n + 4) & ~3) : 0); }
  __host__ __device__ size_t list_at(int list) const {
    size_t at = 8 + 2 * (size_t)((n + 4) & ~3);
    for (int i = 0; i < list; ++i) at += 4 * (size_t)cap(i);
    return at;
  }
  __host__ __device__ size_t bytes() const { return 4 * list_at(LISTS); }
};

// what the kernels read of it
struct RowOrder {
  const int* order;
  const int* offsets;
  const int* tiles;
};

size_t adapter_route_ws_bytes(const RowLists& l);
hipError_t launch_adapter_route(const RowLists& l, const int* adapter, int* order, int* offsets, int* tiles, char* ws,
                                hipStream_t st);

// ---- low-rank updates
struct LowrankDims {
  int T, n, K, N, r;
  bool f32;  // x, y and dx are fp32 (else bf16)
  int n_seg;
  int seg[MAX_SEG];
};
size_t lowrank_ws_bytes(const LowrankDims& d, bool bwd);

struct LowrankPtrs {
  RowOrder rows;
  const void* x;
  const uint16_t* A;
  const uint16_t* B;
  const float* scale;
  const void* y_base;
  void* y;
  float* v;
};
hipError_t launch_lowrank_fwd(const LowrankDims& d, const LowrankPtrs& q, char* ws, hipStream_t st);

struct LowrankGradPtrs {
  RowOrder rows;
  const uint16_t* dy;
  const void* x;
  const float* v;
  const uint16_t* A;
  const uint16_t* B;
  const float* scale;
  const void* dx_base;
  void* dx;
  float* dA;
  float* dB;
};
hipError_t launch_lowrank_bwd(const LowrankDims& d, const LowrankGradPtrs& q, char* ws, hipStream_t st);

// ---- block rotations
struct RotateDims {
  int T, n, N, b;
  bool f32;  // z, y are fp32 (else bf16)
};
size_t rotate_ws_bytes(const RotateDims& d, bool bwd);
hipError_t launch_rotate_fwd(const RotateDims& d, const RowOrder& rows, const void* z, const uint16_t* Rops, void* y,
                             hipStream_t st);
hipError_t launch_rotate_bwd(const RotateDims& d, const RowOrder& rows, const uint16_t* dy, const void* y,
                             const float* Rf, const uint16_t* Rops, uint16_t* dz, float* dq, char* ws, hipStream_t st);

}  // namespace oft
