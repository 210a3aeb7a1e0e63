// Internal interface of the kernels over vocabulary logits (host side).  The
// C-ABI layer (vocab_abi.cpp) validates every argument before calling these.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace oft {

struct VocabDims {
  int T, V, k;
  long ld, ldg;
  float invtau;
  bool f32;  // logits and d_logits are fp32 (else bf16)
  bool accumulate;
};

size_t vocab_ws_bytes(const VocabDims& d);

struct LogprobPtrs {
  const void* logits;
  const int* labels;
  float* logp;
  float* entropy;
  int* top_idx;
  float* top_logp;
  float* stats;
};
hipError_t launch_token_logprobs(const VocabDims& d, const LogprobPtrs& q, char* ws, hipStream_t st);

struct LogprobGradPtrs {
  const void* logits;
  const int* labels;
  const float* stats;
  const float* entropy;
  const float* g_logp;
  const float* g_entropy;
  void* d_logits;
};
hipError_t launch_token_logprobs_bwd(const VocabDims& d, const LogprobGradPtrs& q, hipStream_t st);

hipError_t launch_distill(const VocabDims& d, const void* logits, const int* idx, const float* teacher, float* loss,
                          float* stats, char* ws, hipStream_t st);
hipError_t launch_distill_bwd(const VocabDims& d, const void* logits, const int* idx, const float* teacher,
                              const float* stats, const float* g_loss, void* d_logits, hipStream_t st);

}  // namespace oft
