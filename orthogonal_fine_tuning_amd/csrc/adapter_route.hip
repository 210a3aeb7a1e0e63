// Rows sorted by the adapter that they use, and the work lists of the
// kernels that run over them (oft_adapter_route in oft.h).
//
// A stable counting sort: each wave takes a contiguous run of rows, keeps
// their adapters in registers and counts them into its own table in LDS, the
// count so far being each row's place among the wave's; a scan over adapters
// and waves turns the tables into first positions.  Rows of a wave with the
// same adapter find each other by one ballot per bit of the adapter number, so
// that nothing depends on the order of atomics.  Up to ONE_WG rows one
// workgroup does it all: the call is a chain of latencies, not of bytes (64
// rows: 4.7 us, an empty launch 2).  More rows are too many instructions for
// one (20011 rows: 24 us): workgroups count a slab of them each, and in a
// second launch each adds up the slabs before it, all of them from the caches.
#include "adapter_device.h"
#include "oft_prof.h"

namespace oft {
namespace {

constexpr int THREADS = 1024, WAVES = THREADS / 64;
constexpr int ONE_WG = 4096, SLABS = 192;
constexpr int FEW = 256;  // rows that four waves take
constexpr int KEYS = MAX_ADAPTERS + 1;  // adapters, and rows without one
static_assert(THREADS >= MAX_ADAPTERS, "the scan takes an adapter a thread");

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

// The rows of one wave, RUN steps of 64, in registers: adapter (n: none, PAST
// behind the last row) and, above KEY_BITS, the place among the wave's rows of
// that adapter (at most 64 RUN).
constexpr int KEY_BITS = 11, PAST = (1 << KEY_BITS) - 1;
template <int RUN>
struct Rows {
  int v[RUN];
  __device__ __forceinline__ int key(int i) const { return v[i] & PAST; }
  __device__ __forceinline__ int place(int i) const { return v[i] >> KEY_BITS; }
};

template <int RUN>
__device__ __forceinline__ void load_rows(const int* __restrict__ adapter, int n, int lo, int hi, Rows<RUN>& r) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < RUN; ++i) {
    const int t = lo + 64 * i + lane;
    r.v[i] = t < hi ? key_of(adapter[t], n) : PAST;
  }
}

template <int RUN>
__device__ __forceinline__ void count_rows(int bits, Rows<RUN>& r, int* table) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < RUN; ++i) {
    const int key = r.key(i);
    const bool on = key != PAST;
    if (__ballot(on) == 0) break;
    const uint64_t m = same_key(key, on, bits);
    const uint64_t below = m & ((1ull << lane) - 1);
    int first = 0;
    if (on && below == 0) first = atomicAdd(&table[key], __popcll(m));
    first = __shfl(first, on ? __ffsll((unsigned long long)m) - 1 : lane);
    r.v[i] = key | ((first + __popcll(below)) << KEY_BITS);
  }
}

// table: the wave's first position of each adapter
template <int RUN>
__device__ __forceinline__ void place_rows(int lo, const Rows<RUN>& r, const int* table, int* __restrict__ order) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < RUN; ++i)
    if (r.key(i) != PAST) order[table[r.key(i)] + r.place(i)] = lo + 64 * i + lane;
}

// The sums over the adapters below each one: its rows, its tiles and pieces,
// its partial slots.
constexpr int SUMS = 7;  // rows, the four lists, partial slots of the two lists of pieces

template <int TH>  // threads, and adapters at most
struct Scan {
  int first[SUMS][TH + 2];
  int wave[SUMS][TH / 64];
};

// total: rows of this thread's adapter -> s.first[0 .. N - 1]
template <int N, int TH>
__device__ __forceinline__ void scan_sums(const RowLists& l, Scan<TH>& s, int total) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = l.n;
  int own[SUMS], sum[SUMS];
  own[0] = tid < n ? total : 0;
  if constexpr (N > 1) {
#pragma unroll
    for (int i = 0; i < LISTS; ++i) own[1 + i] = l.count(i, own[0]);
    own[5] = own[3] >= 2 ? own[3] : 0;
    own[6] = own[4] >= 2 ? own[4] : 0;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    sum[i] = wave_scan(own[i]);
    if (lane == 63) s.wave[i][wave] = sum[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    int before = 0;
#pragma unroll
    for (int w = 0; w < TH / 64; ++w) before += w < wave ? s.wave[i][w] : 0;
    sum[i] += before;
    if (tid < n) s.first[i][tid + 1] = sum[i];
    if (tid == 0) s.first[i][0] = 0;
  }
  __syncthreads();
}

// offsets, the lists and their counts from the sums
template <int TH>
__device__ __forceinline__ void write_lists(const RowLists& l, const Scan<TH>& s, int* __restrict__ offsets,
                                            int* __restrict__ tiles) {
  const int tid = threadIdx.x, n = l.n;
  for (int a = tid; a <= n; a += TH) offsets[a] = s.first[0][a];
  const int rest = l.T - s.first[0][n];  // rows without an adapter
  if (tid < 8) tiles[tid] = tid < LISTS ? s.first[1 + tid][n] + l.count(tid, rest) : 0;
  for (int a = tid; a <= n; a += TH) {
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
  for (int e = tid; e < all; e += TH) {
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

// RUN steps of 64 rows a wave at most; as many waves as have rows count.
template <int RUN, int TH>
__global__ __launch_bounds__(TH) void route_one_kernel(RowLists l, int bits, const int* __restrict__ adapter,
                                                            int* __restrict__ order, int* __restrict__ offsets,
                                                            int* __restrict__ tiles) {
  constexpr int WAVES = TH / 64;
  __shared__ int table[WAVES][TH + 1];
  __shared__ Scan<TH> s;
  const int tid = threadIdx.x, wave = tid >> 6, n = l.n;
  const int per = RUN == 1 ? 64 : ((l.T + WAVES * 64 - 1) / (WAVES * 64)) * 64;  // rows of a wave
  const int waves = (l.T + per - 1) / per;
  const int lo = wave * per, hi = min(l.T, lo + per);
  Rows<RUN> r;
  load_rows<RUN>(adapter, n, lo, hi, r);
  for (int w = 0; w < waves; ++w)
    for (int a = tid; a <= n; a += TH) table[w][a] = 0;
  __syncthreads();
  count_rows<RUN>(bits, r, table[wave]);
  __syncthreads();
  // rows of this thread's adapter, and of the waves before each one
  int total = 0;
  if (tid < n)
    for (int w = 0; w < waves; ++w) {
      const int c = table[w][tid];
      table[w][tid] = total;
      total += c;
    }
  scan_sums<SUMS, TH>(l, s, total);
  if (tid < n)
    for (int w = 0; w < waves; ++w) table[w][tid] += s.first[0][tid];
  if (tid < 64) {  // rows without an adapter, behind all others
    int v = tid < waves ? table[tid][n] : 0;
    v = wave_scan(v) - v;
    if (tid < waves) table[tid][n] = s.first[0][n] + v;
  }
  __syncthreads();
  place_rows<RUN>(lo, r, table[wave], order);
  write_lists(l, s, offsets, tiles);
}

// ---- more rows than one workgroup takes
// RUN steps of 64 rows a wave
template <int RUN>
__global__ __launch_bounds__(THREADS) void route_count_kernel(RowLists l, int bits, const int* __restrict__ adapter,
                                                              int* __restrict__ counts) {
  __shared__ int table[KEYS];
  const int tid = threadIdx.x;
  Rows<RUN> r;
  load_rows<RUN>(adapter, l.n, (blockIdx.x * WAVES + (tid >> 6)) * 64 * RUN, l.T, r);
  for (int a = tid; a <= l.n; a += THREADS) table[a] = 0;
  __syncthreads();
  count_rows<RUN>(bits, r, table);
  __syncthreads();
  for (int a = tid; a <= l.n; a += THREADS) counts[(size_t)blockIdx.x * (l.n + 1) + a] = table[a];
}

template <int RUN>
__global__ __launch_bounds__(THREADS) void route_place_kernel(RowLists l, int bits, const int* __restrict__ adapter,
                                                              const int* __restrict__ counts, int* __restrict__ order,
                                                              int* __restrict__ offsets, int* __restrict__ tiles) {
  __shared__ int table[WAVES][KEYS];
  __shared__ Scan<THREADS> s;
  const int tid = threadIdx.x, wave = tid >> 6, n = l.n;
  const int lo = (blockIdx.x * WAVES + wave) * 64 * RUN;
  Rows<RUN> r;
  load_rows<RUN>(adapter, n, lo, l.T, r);
  // this thread's adapter: rows in all, and in the slabs before this one
  int total = 0, before = 0;
  if (tid < n) {
    const int* c = counts + tid;
#pragma unroll 8
    for (int g = 0; g < (int)gridDim.x; ++g, c += n + 1) {
      total += *c;
      before += g < (int)blockIdx.x ? *c : 0;
    }
  }
  for (int w = 0; w < WAVES; ++w)
    for (int a = tid; a <= n; a += THREADS) table[w][a] = 0;
  __syncthreads();
  count_rows<RUN>(bits, r, table[wave]);
  if (blockIdx.x == 0) scan_sums<SUMS, THREADS>(l, s, total);
  else scan_sums<1, THREADS>(l, s, total);
  if (tid < n) {
    int at = s.first[0][tid] + before;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      const int c = table[w][tid];
      table[w][tid] = at;
      at += c;
    }
  }
  if (wave == 0) {  // rows without an adapter, behind all others
    int at = 0;
    for (int g = tid; g < (int)blockIdx.x; g += 64) at += counts[(size_t)g * (n + 1) + n];
    at = __shfl(wave_scan(at), 63);
    int v = tid < WAVES ? table[tid][n] : 0;
    v = wave_scan(v) - v;
    if (tid < WAVES) table[tid][n] = s.first[0][n] + at + v;
  }
  __syncthreads();
  place_rows<RUN>(lo, r, table[wave], order);
  if (blockIdx.x == 0) write_lists(l, s, offsets, tiles);
}

// Steps of 64 rows a wave takes: one while that gives SLABS workgroups at
// most, else eight, so that each has fewer slabs to add up (300 adapters, us:
// 131072 rows 18.5 and 25.2, 196608 21.4 and 26.7, 262144 28 with either).
int slab_rows(int T) { return T <= SLABS * THREADS ? THREADS : 8 * THREADS; }
int slabs_of(int T) { return (T + slab_rows(T) - 1) / slab_rows(T); }

}  // namespace

size_t adapter_route_ws_bytes(const RowLists& l) { return l.T <= ONE_WG ? 0 : 4 * (size_t)slabs_of(l.T) * (l.n + 1); }

hipError_t launch_adapter_route(const RowLists& l, const int* adapter, int* order, int* offsets, int* tiles, char* ws,
                                hipStream_t st) {
  ProfScope prof(st, "adapter.route");
  int bits = 0;
  while ((1 << bits) <= l.n) ++bits;
  if (l.T <= ONE_WG) {
    auto run = [&](auto steps, auto threads) {
      constexpr int TH = decltype(threads)::value;
      hipLaunchKernelGGL((route_one_kernel<decltype(steps)::value, TH>), dim3(1), dim3(TH), 0, st, l, bits, adapter, order,
                         offsets, tiles);
    };
    using std::integral_constant;
    // decoded rows of few adapters: four waves' barriers (64 rows, 64 adapters
    // 4.7 us, 5.7 with sixteen; 256 rows, 128 adapters 5.9 and 6.1, 256 of both 7.0 and 6.4)
    if (l.T <= FEW && l.n <= FEW / 2) run(integral_constant<int, 1>{}, integral_constant<int, FEW>{});
    else if (l.T <= THREADS) run(integral_constant<int, 1>{}, integral_constant<int, THREADS>{});
    else run(integral_constant<int, ONE_WG / THREADS>{}, integral_constant<int, THREADS>{});
    return hipGetLastError();
  }
  int* counts = reinterpret_cast<int*>(ws);
  auto run = [&](auto steps) {
    constexpr int RUN = decltype(steps)::value;
    const int slabs = slabs_of(l.T);
    hipLaunchKernelGGL(route_count_kernel<RUN>, dim3(slabs), dim3(THREADS), 0, st, l, bits, adapter, counts);
    hipLaunchKernelGGL(route_place_kernel<RUN>, dim3(slabs), dim3(THREADS), 0, st, l, bits, adapter, counts, order,
                       offsets, tiles);
  };
  if (slab_rows(l.T) == THREADS) run(std::integral_constant<int, 1>{});
  else run(std::integral_constant<int, 8>{});
  return hipGetLastError();
}

}  // namespace oft
