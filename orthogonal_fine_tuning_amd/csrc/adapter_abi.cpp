// extern "C" entry points of the operators on adapters of many requests
// (declared in include/oft.h).  Arguments are validated on the host before
// anything is enqueued.
#include <hip/hip_runtime.h>

#include "oft.h"
#include "oft_adapter.h"
#include "oft_launch.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ptr_ok(const void* p) { return p != nullptr && aligned16(p); }
bool opt_ok(const void* p) { return p == nullptr || aligned16(p); }

int32_t hip_status(hipError_t e) {
  if (e == hipSuccess) return OFT_OK;
  oft::set_last_hip_error(static_cast<int>(e));
  return OFT_EHIP;
}

static_assert(oft::MAX_ADAPTERS == OFT_MAX_ADAPTERS && oft::MAX_SEG == OFT_MAX_SEGMENTS, "limits are the ABI's");

int32_t validate_counts(int32_t T, int32_t n) {
  if (T < 0 || n < 1) return OFT_EINVAL;
  return T > (1 << 22) || n > OFT_MAX_ADAPTERS ? OFT_EUNSUPPORTED : OFT_OK;
}

// A launch has fewer than 2^32 threads along its grid's x dimension, where
// tiles of 64 rows and 64 columns (and one unfull row tile per adapter) lie: a
// wave each, 2^28 threads at this limit.
bool elements_ok(int32_t T, int32_t cols) { return (int64_t)T * cols <= (1LL << 34); }

int32_t validate_lowrank(const oft_lowrank_desc* d) {
  if (d == nullptr) return OFT_EINVAL;
  if (d->K <= 0 || d->N <= 0 || d->r <= 0) return OFT_EINVAL;
  const int32_t v = validate_counts(d->T, d->n);
  if (v != OFT_OK) return v;
  if (d->K > (1 << 20) || d->N > (1 << 20) || d->r > OFT_MAX_RANK) return OFT_EUNSUPPORTED;
  if (!elements_ok(d->T, d->K) || !elements_ok(d->T, d->N)) return OFT_EUNSUPPORTED;
  if (d->dtype != OFT_DT_BF16 && d->dtype != OFT_DT_F32) return OFT_EDTYPE;
  if (d->n_seg < 1 || d->n_seg > OFT_MAX_SEGMENTS) return OFT_EUNSUPPORTED;
  long long sum = 0;
  for (int s = 0; s < d->n_seg; ++s) {
    if (d->seg[s] <= 0 || d->seg[s] % 16 != 0) return OFT_ESHAPE;
    sum += d->seg[s];
  }
  if (sum != d->N || d->K % 64 != 0 || d->r % 8 != 0) return OFT_ESHAPE;
  return OFT_OK;
}

oft::LowrankDims dims(const oft_lowrank_desc* d) {
  oft::LowrankDims o{d->T, d->n, d->K, d->N, d->r, d->dtype == OFT_DT_F32, d->n_seg, {}};
  for (int s = 0; s < d->n_seg; ++s) o.seg[s] = d->seg[s];
  return o;
}

int32_t validate_rotate(const oft_rotate_desc* d) {
  if (d == nullptr || d->N <= 0) return OFT_EINVAL;
  const int32_t v = validate_counts(d->T, d->n);
  if (v != OFT_OK) return v;
  if (d->N > (1 << 20) || !elements_ok(d->T, d->N)) return OFT_EUNSUPPORTED;
  if (d->dtype != OFT_DT_BF16 && d->dtype != OFT_DT_F32) return OFT_EDTYPE;
  if (d->b != 16 && d->b != 32) return OFT_EUNSUPPORTED;
  return d->N % 32 != 0 ? OFT_ESHAPE : OFT_OK;
}

oft::RotateDims dims(const oft_rotate_desc* d) {
  return oft::RotateDims{d->T, d->n, d->N, d->b, d->dtype == OFT_DT_F32};
}

int32_t rows_ok(const oft_adapter_rows* rows, int32_t T, int32_t n) {
  if (rows == nullptr) return OFT_EINVAL;
  if (rows->T != T || rows->n != n) return OFT_ESHAPE;
  if (T > 0 && !ptr_ok(rows->order)) return OFT_EINVAL;
  return ptr_ok(rows->offsets) && ptr_ok(rows->tiles) ? OFT_OK : OFT_EINVAL;
}
oft::RowOrder order_of(const oft_adapter_rows* rows) { return oft::RowOrder{rows->order, rows->offsets, rows->tiles}; }

int32_t ws_ok(size_t need, const void* ws, size_t ws_bytes) {
  if (need == 0) return OFT_OK;
  if (!ptr_ok(ws)) return OFT_EINVAL;
  return ws_bytes < need ? OFT_EWORKSPACE : OFT_OK;
}

// address ranges of a and b bytes
bool apart(const void* p, size_t a, const void* q, size_t b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(p), y = reinterpret_cast<uintptr_t>(q);
  return p == nullptr || q == nullptr || x + a <= y || y + b <= x;
}
bool same_or_apart(const void* p, const void* q, size_t bytes) { return p == q || apart(p, bytes, q, bytes); }

}  // namespace

extern "C" {

int32_t oft_adapter_rows_bytes(int32_t T, int32_t n, size_t* tiles_bytes, size_t* ws_bytes) {
  if (tiles_bytes == nullptr || ws_bytes == nullptr) return OFT_EINVAL;
  const int32_t v = validate_counts(T, n);
  if (v != OFT_OK) return v;
  const oft::RowLists l{T, n};
  *tiles_bytes = l.bytes();
  *ws_bytes = oft::adapter_route_ws_bytes(l);
  return OFT_OK;
}

int32_t oft_adapter_route(const int32_t* adapter, const oft_adapter_rows* rows, void* ws, size_t ws_bytes,
                          void* stream) {
  if (rows == nullptr) return OFT_EINVAL;
  int32_t v = validate_counts(rows->T, rows->n);
  if (v != OFT_OK) return v;
  if ((v = rows_ok(rows, rows->T, rows->n)) != OFT_OK) return v;
  if (rows->T > 0 && !ptr_ok(adapter)) return OFT_EINVAL;
  const oft::RowLists l{rows->T, rows->n};
  if ((v = ws_ok(oft::adapter_route_ws_bytes(l), ws, ws_bytes)) != OFT_OK) return v;
  return hip_status(oft::launch_adapter_route(l, adapter, rows->order, rows->offsets, rows->tiles,
                                              static_cast<char*>(ws), static_cast<hipStream_t>(stream)));
}

int32_t oft_lowrank_workspace_bytes(const oft_lowrank_desc* d, int32_t pass, size_t* bytes) {
  if (bytes == nullptr || (pass != OFT_PASS_FWD && pass != OFT_PASS_BWD)) return OFT_EINVAL;
  const int32_t v = validate_lowrank(d);
  if (v != OFT_OK) return v;
  *bytes = d->T == 0 ? 0 : oft::lowrank_ws_bytes(dims(d), pass == OFT_PASS_BWD);
  return OFT_OK;
}

int32_t oft_lowrank_fwd(const oft_lowrank_desc* d, const oft_adapter_rows* rows, const void* x, const uint16_t* A,
                        const uint16_t* B, const float* scale, const void* y_base, void* y, float* v_or_null, void* ws,
                        size_t ws_bytes, void* stream) {
  int32_t v = validate_lowrank(d);
  if (v != OFT_OK) return v;
  if (d->T == 0) return OFT_OK;
  if ((v = rows_ok(rows, d->T, d->n)) != OFT_OK) return v;
  if (!ptr_ok(x) || !ptr_ok(A) || !ptr_ok(B) || !ptr_ok(scale) || !ptr_ok(y_base) || !ptr_ok(y) || !opt_ok(v_or_null))
    return OFT_EINVAL;
  const size_t size = d->dtype == OFT_DT_F32 ? 4 : 2, T = (size_t)d->T;
  if (!same_or_apart(y, y_base, T * d->N * size) || !apart(y, T * d->N * size, x, T * d->K * size)) return OFT_EINVAL;
  const oft::LowrankDims o = dims(d);
  if ((v = ws_ok(oft::lowrank_ws_bytes(o, false), ws, ws_bytes)) != OFT_OK) return v;
  const oft::LowrankPtrs q{order_of(rows), x, A, B, scale, y_base, y, v_or_null};
  return hip_status(oft::launch_lowrank_fwd(o, q, static_cast<char*>(ws), static_cast<hipStream_t>(stream)));
}

int32_t oft_lowrank_bwd(const oft_lowrank_desc* d, const oft_adapter_rows* rows, const uint16_t* dy, const void* x,
                        const float* v_saved, const uint16_t* A, const uint16_t* B, const float* scale,
                        const void* dx_base_or_null, void* dx_or_null, float* dA_or_null, float* dB_or_null, void* ws,
                        size_t ws_bytes, void* stream) {
  int32_t v = validate_lowrank(d);
  if (v != OFT_OK) return v;
  if ((v = rows_ok(rows, d->T, d->n)) != OFT_OK) return v;
  if (!opt_ok(dx_base_or_null) || !opt_ok(dx_or_null) || !opt_ok(dA_or_null) || !opt_ok(dB_or_null)) return OFT_EINVAL;
  const bool dx = dx_or_null != nullptr, dA = dA_or_null != nullptr, dB = dB_or_null != nullptr;
  if (!dx && !dA && !dB) return OFT_OK;
  const oft::LowrankDims o = dims(d);
  if (d->T > 0) {
    // what a gradient reads has to be there: dy for all, x for dA, v for dB
    if (!ptr_ok(dy) || !ptr_ok(scale) || !opt_ok(x) || !opt_ok(v_saved) || !opt_ok(A) || !opt_ok(B)) return OFT_EINVAL;
    if ((dA && x == nullptr) || (dB && v_saved == nullptr) || (dx && A == nullptr) || ((dx || dA) && B == nullptr))
      return OFT_EINVAL;
    const size_t size = d->dtype == OFT_DT_F32 ? 4 : 2, T = (size_t)d->T;
    const size_t row_bytes = T * d->K * size;
    if (dx && ((dx_base_or_null != nullptr && !same_or_apart(dx_or_null, dx_base_or_null, row_bytes)) ||
               !apart(dx_or_null, row_bytes, dy, T * d->N * 2) || !apart(dx_or_null, row_bytes, x, row_bytes)))
      return OFT_EINVAL;
    if ((v = ws_ok(oft::lowrank_ws_bytes(o, true), ws, ws_bytes)) != OFT_OK) return v;
  }
  const oft::LowrankGradPtrs q{order_of(rows), dy, x,          v_saved,    A, B, scale, dx_base_or_null,
                               dx_or_null,     dA_or_null, dB_or_null};
  return hip_status(oft::launch_lowrank_bwd(o, q, static_cast<char*>(ws), static_cast<hipStream_t>(stream)));
}

int32_t oft_rotate_workspace_bytes(const oft_rotate_desc* d, int32_t pass, size_t* bytes) {
  if (bytes == nullptr || (pass != OFT_PASS_FWD && pass != OFT_PASS_BWD)) return OFT_EINVAL;
  const int32_t v = validate_rotate(d);
  if (v != OFT_OK) return v;
  *bytes = d->T == 0 ? 0 : oft::rotate_ws_bytes(dims(d), pass == OFT_PASS_BWD);
  return OFT_OK;
}

int32_t oft_rotate_fwd(const oft_rotate_desc* d, const oft_adapter_rows* rows, const void* z, const uint16_t* R_ops,
                       void* y, void* stream) {
  int32_t v = validate_rotate(d);
  if (v != OFT_OK) return v;
  if (d->T == 0) return OFT_OK;
  if ((v = rows_ok(rows, d->T, d->n)) != OFT_OK) return v;
  if (!ptr_ok(z) || !ptr_ok(R_ops) || !ptr_ok(y)) return OFT_EINVAL;
  if (!same_or_apart(y, z, (size_t)d->T * d->N * (d->dtype == OFT_DT_F32 ? 4 : 2))) return OFT_EINVAL;
  return hip_status(oft::launch_rotate_fwd(dims(d), order_of(rows), z, R_ops, y, static_cast<hipStream_t>(stream)));
}

int32_t oft_rotate_bwd(const oft_rotate_desc* d, const oft_adapter_rows* rows, const uint16_t* dy, const void* y_saved,
                       const float* R_f32, const uint16_t* R_ops, uint16_t* dz_or_null, float* dq_or_null, void* ws,
                       size_t ws_bytes, void* stream) {
  int32_t v = validate_rotate(d);
  if (v != OFT_OK) return v;
  if ((v = rows_ok(rows, d->T, d->n)) != OFT_OK) return v;
  if (!opt_ok(dz_or_null) || !opt_ok(dq_or_null)) return OFT_EINVAL;
  const bool dz = dz_or_null != nullptr, dq = dq_or_null != nullptr;
  if (!dz && !dq) return OFT_OK;
  if (d->T == 0 && !dq) return OFT_OK;
  const oft::RotateDims o = dims(d);
  if (d->T > 0) {
    if (!ptr_ok(dy) || !opt_ok(y_saved) || !opt_ok(R_f32) || !opt_ok(R_ops)) return OFT_EINVAL;
    if ((dq && (y_saved == nullptr || R_f32 == nullptr)) || (dz && R_ops == nullptr)) return OFT_EINVAL;
    const size_t elems = (size_t)d->T * d->N;
    if (dz && (!same_or_apart(dz_or_null, dy, 2 * elems) ||
               !apart(dz_or_null, 2 * elems, y_saved, elems * (o.f32 ? 4 : 2))))
      return OFT_EINVAL;
    if (dq && (v = ws_ok(oft::rotate_ws_bytes(o, true), ws, ws_bytes)) != OFT_OK) return v;
  }
  return hip_status(oft::launch_rotate_bwd(o, order_of(rows), dy, y_saved, R_f32, R_ops, dz_or_null, dq_or_null,
                                           static_cast<char*>(ws), static_cast<hipStream_t>(stream)));
}

}  // extern "C"
