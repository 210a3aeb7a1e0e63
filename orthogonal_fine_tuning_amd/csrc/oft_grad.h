// Internal interface of the gradient norm and clipping (host side).  The
// C-ABI layer (grad_abi.cpp) validates every argument before calling these.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace oft {

struct GradList {
  int m;
  const void* const* grads;
  const int64_t* numel;
  bool f32;  // else bf16
};
size_t grad_ws_bytes(int m, const int64_t* numel);
hipError_t launch_grad_sumsq(const GradList& l, double* sumsq, char* ws, hipStream_t st);
hipError_t launch_grad_clip(const GradList& l, const double* sumsq, float max_norm, void* const* out, float* stats,
                            hipStream_t st);

}  // namespace oft
