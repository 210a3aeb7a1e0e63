// extern "C" entry points of the gradient norm and clipping (declared in
// include/oft.h).  Arguments are validated on the host before anything is
// enqueued.
#include <hip/hip_runtime.h>

#include "oft.h"
#include "oft_grad.h"
#include "oft_launch.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

uintptr_t size_of(int32_t dtype) { return dtype == OFT_DT_F32 ? 4 : 2; }

int32_t validate_sizes(int32_t m, const int64_t* numel, int32_t dtype) {
  if (m < 0 || (m > 0 && numel == nullptr)) return OFT_EINVAL;
  if (dtype != OFT_DT_BF16 && dtype != OFT_DT_F32) return OFT_EDTYPE;
  if (m > OFT_MAX_GRADS) return OFT_EUNSUPPORTED;
  int64_t total = 0;
  for (int32_t i = 0; i < m; ++i) {
    if (numel[i] < 0) return OFT_EINVAL;
    // (each below 2^36 and at most 2^16 of them: the sum stays inside 64 bits)
    if (numel[i] >= (1LL << 36)) return OFT_EUNSUPPORTED;
    total += numel[i];
  }
  // a workgroup of 256 threads takes 16384 elements, and a launch has fewer
  // than 2^32 threads
  return total >= (1LL << 36) ? OFT_EUNSUPPORTED : OFT_OK;
}

int32_t validate_list(int32_t m, const void* const* grads, const int64_t* numel, int32_t dtype) {
  const int32_t v = validate_sizes(m, numel, dtype);
  if (v != OFT_OK) return v;
  if (m > 0 && grads == nullptr) return OFT_EINVAL;
  for (int32_t i = 0; i < m; ++i)
    if (numel[i] > 0 && !aligned(grads[i], size_of(dtype))) return OFT_EINVAL;
  return OFT_OK;
}

int32_t hip_status(hipError_t e) {
  if (e == hipSuccess) return OFT_OK;
  oft::set_last_hip_error(static_cast<int>(e));
  return OFT_EHIP;
}

}  // namespace

extern "C" {

int32_t oft_grad_workspace_bytes(int32_t m, const int64_t* numel, int32_t dtype, size_t* bytes) {
  if (bytes == nullptr) return OFT_EINVAL;
  const int32_t v = validate_sizes(m, numel, dtype);
  if (v != OFT_OK) return v;
  *bytes = oft::grad_ws_bytes(m, numel);
  return OFT_OK;
}

int32_t oft_grad_sumsq(int32_t m, const void* const* grads, const int64_t* numel, int32_t dtype, double* sumsq,
                       void* ws, size_t ws_bytes, void* stream) {
  const int32_t v = validate_list(m, grads, numel, dtype);
  if (v != OFT_OK) return v;
  if (!aligned(sumsq, 8)) return OFT_EINVAL;
  const size_t need = oft::grad_ws_bytes(m, numel);
  if (need > 0 && !aligned(ws, 16)) return OFT_EINVAL;
  if (ws_bytes < need) return OFT_EWORKSPACE;
  const oft::GradList l{m, grads, numel, dtype == OFT_DT_F32};
  return hip_status(oft::launch_grad_sumsq(l, sumsq, static_cast<char*>(ws), static_cast<hipStream_t>(stream)));
}

int32_t oft_grad_clip(int32_t m, const void* const* grads, const int64_t* numel, int32_t dtype, const double* sumsq,
                      float max_norm, void* const* out, float* stats, void* stream) {
  const int32_t v = validate_list(m, grads, numel, dtype);
  if (v != OFT_OK) return v;
  if (!(max_norm >= 0.0f)) return OFT_EINVAL;  // (NaN fails the comparison)
  if (!aligned(sumsq, 8) || !aligned(stats, 8)) return OFT_EINVAL;
  if (m > 0 && out == nullptr) return OFT_EINVAL;
  const uintptr_t size = size_of(dtype);
  for (int32_t i = 0; i < m; ++i) {
    if (numel[i] == 0) continue;
    if (!aligned(out[i], size)) return OFT_EINVAL;
    // a gradient's output is the gradient itself or apart from it
    const uintptr_t a = reinterpret_cast<uintptr_t>(grads[i]), b = reinterpret_cast<uintptr_t>(out[i]);
    const uintptr_t len = (uintptr_t)numel[i] * size;
    if (a != b && a < b + len && b < a + len) return OFT_EINVAL;
  }
  const oft::GradList l{m, grads, numel, dtype == OFT_DT_F32};
  return hip_status(oft::launch_grad_clip(l, sumsq, max_norm, out, stats, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
