// Rows sorted by the adapter that they use, and the work lists of the
// kernels that run over them (oft_adapter_route in oft.h).
//
// A stable counting sort: each wave counts the adapters of a contiguous run
// of rows into its own table in LDS, the tables become first positions by a
// scan over adapters and waves, and each wave walks its rows again, in order,
// to hand out positions.  Rows of a wave with the same adapter find each
// other by one ballot per bit of the adapter number, so that nothing depends
// on the order of atomics.  Up to ONE_WG rows one workgroup does it all (the
// call is a chain of latencies, not of bytes); above, workgroups of SLAB rows
// count and scatter, with a scan by one workgroup between.
#include "adapter_device.h"
#include "oft_prof.h"

namespace oft {
namespace {

constexpr int THREADS = 1024, WAVES = THREADS / 64;
constexpr int ONE_WG = 16384, SLAB = 8192;
constexpr int KEYS = MAX_ADAPTERS + 1;  // adapters, and rows without one

__device__ __forceinline__ int key_of(int a, int n) { return (unsigned)a < (unsigned)n ? a : n; }

// inclusive sum over the lanes up to this one
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);  // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);  // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);  // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1, 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2, 3
  return v;
}

// lanes whose key is this lane's (lanes without `on` match none)
__device__ __forceinline__ uint64_t same_key(int key, bool on, int bits) {
  uint64_t m = __ballot(on);
  for (int b = 0; b < bits; ++b) {
    const bool set = (key >> b) & 1;
    const uint64_t s = __ballot(set);
    m &= set ? s : ~s;
  }
  return m;
}

// rows of one wave: [lo, hi)
struct Run {
  int lo, hi;
};
__device__ __forceinline__ Run wave_run(int lo, int hi, int wave) {
  const int per = ((hi - lo + WAVES * 64 - 1) / (WAVES * 64)) * 64;
  const int a = min(hi, lo + wave * per);
  return Run{a, min(hi, a + per)};
}

__device__ __forceinline__ void count_rows(const int* __restrict__ adapter, int n, int bits, Run run, int* table) {
  const int lane = threadIdx.x & 63;
  for (int i = run.lo; i < run.hi; i += 64) {
    const bool on = i + lane < run.hi;
    const int key = on ? key_of(adapter[i + lane], n) : 0;
    const uint64_t m = same_key(key, on, bits);
    if (on && (m & ((1ull << lane) - 1)) == 0) atomicAdd(&table[key], __popcll(m));
  }
}

__device__ __forceinline__ void place_rows(const int* __restrict__ adapter, int n, int bits, Run run, int* table,
                                           int* __restrict__ order) {
  const int lane = threadIdx.x & 63;
  for (int i = run.lo; i < run.hi; i += 64) {
    const bool on = i + lane < run.hi;
    const int key = on ? key_of(adapter[i + lane], n) : 0;
    const uint64_t m = same_key(key, on, bits);
    const uint64_t below = m & ((1ull << lane) - 1);
    int first = 0;
    if (on && below == 0) first = atomicAdd(&table[key], __popcll(m));
    first = __shfl(first, on ? __ffsll((unsigned long long)m) - 1 : lane);
    if (on) order[first + __popcll(below)] = i + lane;
  }
}

// The sums over the adapters below each one: its rows, its tiles and pieces,
// its partial slots.
constexpr int SUMS = 7;  // rows, the four lists, partial slots of the two lists of pieces

struct Scan {
  int first[SUMS][KEYS + 1];
  int wave[SUMS][WAVES];
};

// total[a]: rows of adapter a.  Writes offsets, the lists and their counts.
__device__ __forceinline__ void scan_and_list(const RowLists& l, Scan& s, int total, int* __restrict__ offsets,
                                              int* __restrict__ tiles) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = l.n;
  int own[SUMS], sum[SUMS];
  own[0] = tid < n ? total : 0;
#pragma unroll
  for (int i = 0; i < LISTS; ++i) own[1 + i] = l.count(i, own[0]);
  own[5] = own[3] >= 2 ? own[3] : 0;
  own[6] = own[4] >= 2 ? own[4] : 0;
#pragma unroll
  for (int i = 0; i < SUMS; ++i) {
    sum[i] = wave_scan(own[i]);
    if (lane == 63) s.wave[i][wave] = sum[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < SUMS; ++i) {
    int before = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) before += w < wave ? s.wave[i][w] : 0;
    sum[i] += before;
    if (tid < n) s.first[i][tid + 1] = sum[i];
    if (tid == 0) s.first[i][0] = 0;
  }
  __syncthreads();
  if (tid < n) offsets[tid + 1] = sum[0];
  if (tid == 0) offsets[0] = 0;
  const int rest = l.T - s.first[0][n];  // rows without an adapter
  if (tid < 8) tiles[tid] = tid < LISTS ? s.first[1 + tid][n] + l.count(tid, rest) : 0;
  for (int a = tid; a <= n; a += THREADS) {
    tiles[l.part_at(LIST_LONG) + a] = s.first[5][a];
    tiles[l.part_at(LIST_SHORT) + a] = s.first[6][a];
  }
  // all lists in one go, a thread per entry
  int end[LISTS], all = 0;
#pragma unroll
  for (int i = 0; i < LISTS; ++i) {
    all += s.first[1 + i][n] + l.count(i, rest);
    end[i] = all;
  }
  for (int e = tid; e < all; e += THREADS) {
    int list = 0;
#pragma unroll
    for (int i = 0; i + 1 < LISTS; ++i) list += e >= end[i];
    const int t = e - (list == 0 ? 0 : list == 1 ? end[0] : list == 2 ? end[1] : end[2]);
    const int* first = s.first[1 + list];
    int lo = 0, hi = n;  // the adapter (n: none) with first[lo] <= t < first[lo + 1]
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    const int c = l.rows_of(list), at = (t - first[lo]) * c;
    const int rows = lo < n ? s.first[0][lo + 1] - s.first[0][lo] : rest;
    int slot = -1;
    if (list >= LIST_LONG && lo < n && rows > c) slot = s.first[3 + list][lo] + t - first[lo];
    *reinterpret_cast<int4*>(tiles + l.list_at(list) + 4 * (size_t)t) =
        make_int4(lo < n ? lo : -1, s.first[0][lo] + at, min(c, rows - at), slot);
  }
}

__global__ __launch_bounds__(THREADS) void route_one_kernel(RowLists l, int bits, const int* __restrict__ adapter,
                                                            int* __restrict__ order, int* __restrict__ offsets,
                                                            int* __restrict__ tiles) {
  __shared__ int table[WAVES][KEYS];
  __shared__ Scan s;
  const int tid = threadIdx.x, wave = tid >> 6;
  for (int i = tid; i < WAVES * KEYS; i += THREADS) (&table[0][0])[i] = 0;
  __syncthreads();
  const Run run = wave_run(0, l.T, wave);
  count_rows(adapter, l.n, bits, run, table[wave]);
  __syncthreads();
  // rows of this thread's adapter, and of the waves before each one
  int total = 0;
  if (tid < l.n) {
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const int c = table[w][tid];
      table[w][tid] = total;
      total += c;
    }
  }
  scan_and_list(l, s, total, offsets, tiles);
  // (the scan's barriers stand between its writes of s.first and these reads)
  for (int a = tid; a < l.n; a += THREADS) {
#pragma unroll
    for (int w = 0; w < WAVES; ++w) table[w][a] += s.first[0][a];
  }
  if (tid < 64) {  // rows without an adapter, behind all others
    int v = tid < WAVES ? table[tid][l.n] : 0;
    v = wave_scan(v) - v;
    if (tid < WAVES) table[tid][l.n] = s.first[0][l.n] + v;
  }
  __syncthreads();
  place_rows(adapter, l.n, bits, run, table[wave], order);
}

// ---- more rows than one workgroup takes
__global__ __launch_bounds__(THREADS) void route_count_kernel(RowLists l, int bits, const int* __restrict__ adapter,
                                                              int* __restrict__ counts) {
  __shared__ int table[KEYS];
  const int tid = threadIdx.x;
  for (int i = tid; i < KEYS; i += THREADS) table[i] = 0;
  __syncthreads();
  const int lo = blockIdx.x * SLAB;
  count_rows(adapter, l.n, bits, wave_run(lo, min(l.T, lo + SLAB), tid >> 6), table);
  __syncthreads();
  for (int a = tid; a <= l.n; a += THREADS) counts[(size_t)blockIdx.x * (l.n + 1) + a] = table[a];
}

// counts[slab][adapter] -> the slab's first position of the adapter
__global__ __launch_bounds__(THREADS) void route_scan_kernel(RowLists l, int slabs, int* __restrict__ counts,
                                                             int* __restrict__ offsets, int* __restrict__ tiles) {
  __shared__ Scan s;
  const int tid = threadIdx.x, n = l.n;
  int total = 0;
  if (tid < n)
    for (int g = 0; g < slabs; ++g) total += counts[(size_t)g * (n + 1) + tid];
  scan_and_list(l, s, total, offsets, tiles);
  for (int a = tid; a <= n; a += THREADS) {
    int at = s.first[0][a];
    for (int g = 0; g < slabs; ++g) {
      const size_t i = (size_t)g * (n + 1) + a;
      const int c = counts[i];
      counts[i] = at;
      at += c;
    }
  }
}

__global__ __launch_bounds__(THREADS) void route_place_kernel(RowLists l, int bits, const int* __restrict__ adapter,
                                                              const int* __restrict__ first,
                                                              int* __restrict__ order) {
  __shared__ int table[WAVES][KEYS];
  const int tid = threadIdx.x, wave = tid >> 6;
  for (int i = tid; i < WAVES * KEYS; i += THREADS) (&table[0][0])[i] = 0;
  __syncthreads();
  const int lo = blockIdx.x * SLAB;
  const Run run = wave_run(lo, min(l.T, lo + SLAB), wave);
  count_rows(adapter, l.n, bits, run, table[wave]);
  __syncthreads();
  for (int a = tid; a <= l.n; a += THREADS) {
    int at = first[(size_t)blockIdx.x * (l.n + 1) + a];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const int c = table[w][a];
      table[w][a] = at;
      at += c;
    }
  }
  __syncthreads();
  place_rows(adapter, l.n, bits, run, table[wave], order);
}

int slabs_of(const RowLists& l) { return (l.T + SLAB - 1) / SLAB; }

}  // namespace

size_t adapter_route_ws_bytes(const RowLists& l) {
  return l.T <= ONE_WG ? 0 : 4 * (size_t)slabs_of(l) * (l.n + 1);
}

hipError_t launch_adapter_route(const RowLists& l, const int* adapter, int* order, int* offsets, int* tiles, char* ws,
                                hipStream_t st) {
  ProfScope prof(st, "adapter.route");
  int bits = 0;
  while ((1 << bits) <= l.n) ++bits;
  if (l.T <= ONE_WG) {
    hipLaunchKernelGGL(route_one_kernel, dim3(1), dim3(THREADS), 0, st, l, bits, adapter, order, offsets, tiles);
    return hipGetLastError();
  }
  const int slabs = slabs_of(l);
  int* counts = reinterpret_cast<int*>(ws);
  hipLaunchKernelGGL(route_count_kernel, dim3(slabs), dim3(THREADS), 0, st, l, bits, adapter, counts);
  hipLaunchKernelGGL(route_scan_kernel, dim3(1), dim3(THREADS), 0, st, l, slabs, counts, offsets, tiles);
  hipLaunchKernelGGL(route_place_kernel, dim3(slabs), dim3(THREADS), 0, st, l, bits, adapter, counts, order);
  return hipGetLastError();
}

}  // namespace oft
