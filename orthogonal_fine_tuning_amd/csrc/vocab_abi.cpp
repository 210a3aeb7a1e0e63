// extern "C" entry points of the losses on vocabulary logits (declared in
// include/oft.h).  Arguments are validated on the host before anything is
// enqueued.
#include <hip/hip_runtime.h>

#include "oft.h"
#include "oft_launch.h"
#include "oft_vocab.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ptr_ok(const void* p) { return p != nullptr && aligned16(p); }
bool opt_ok(const void* p) { return p == nullptr || aligned16(p); }

// logits and d_logits: rows may start anywhere their type may
bool rows_ok(const oft_vocab_desc* d, const void* p) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (d->dtype == OFT_DT_F32 ? 3u : 1u)) == 0;
}

int32_t validate_vocab(const oft_vocab_desc* d) {
  if (d == nullptr) return OFT_EINVAL;
  if (d->T < 0 || d->V < 1 || d->ld < d->V || d->ld_grad < d->V) return OFT_EINVAL;
  if (d->accumulate != 0 && d->accumulate != 1) return OFT_EINVAL;
  // (a NaN temperature fails the comparison)
  if (!(d->temperature >= 0x1p-20f && d->temperature <= 0x1p20f)) return OFT_EINVAL;
  if (d->dtype != OFT_DT_BF16 && d->dtype != OFT_DT_F32) return OFT_EDTYPE;
  // a backward workgroup takes 2048 elements or more of a row: at most 2^24 of
  // them, what a launch can hold of 256 threads each
  if (d->T > (1 << 22) || d->V > (1 << 24) || (int64_t)d->T * d->V > (1LL << 34)) return OFT_EUNSUPPORTED;
  // (the first two comparisons keep the products inside 64 bits)
  if (d->ld >= (1LL << 40) || d->ld_grad >= (1LL << 40)) return OFT_EUNSUPPORTED;
  if (d->T * d->ld >= (1LL << 40) || d->T * d->ld_grad >= (1LL << 40)) return OFT_EUNSUPPORTED;
  return OFT_OK;
}

int32_t validate_top(const oft_vocab_desc* d) {
  const int32_t v = validate_vocab(d);
  if (v != OFT_OK) return v;
  if (d->k < 0 || d->k > OFT_MAX_TOP) return OFT_EUNSUPPORTED;
  return d->k > d->V ? OFT_ESHAPE : OFT_OK;
}

int32_t validate_teacher(const oft_vocab_desc* d) {
  const int32_t v = validate_vocab(d);
  if (v != OFT_OK) return v;
  return d->k < 1 || d->k > OFT_MAX_TEACHER ? OFT_EUNSUPPORTED : OFT_OK;
}

oft::VocabDims dims(const oft_vocab_desc* d) {
  return oft::VocabDims{d->T,  d->V, d->k, d->ld, d->ld_grad, 1.0f / d->temperature, d->dtype == OFT_DT_F32,
                        d->accumulate == 1};
}

// d_logits apart from logits, or the very same rows
bool grad_rows_ok(const oft_vocab_desc* d, const void* logits, const void* grad) {
  if (logits == grad) return d->ld == d->ld_grad && d->accumulate == 0;
  const uintptr_t size = d->dtype == OFT_DT_F32 ? 4 : 2;
  const uintptr_t a = reinterpret_cast<uintptr_t>(logits), b = reinterpret_cast<uintptr_t>(grad);
  const uintptr_t na = ((uintptr_t)(d->T - 1) * (uintptr_t)d->ld + (uintptr_t)d->V) * size;
  const uintptr_t nb = ((uintptr_t)(d->T - 1) * (uintptr_t)d->ld_grad + (uintptr_t)d->V) * size;
  return a + na <= b || b + nb <= a;
}

int32_t ws_ok(const oft_vocab_desc* d, const void* ws, size_t ws_bytes) {
  const size_t need = oft::vocab_ws_bytes(dims(d));
  if (need == 0) return OFT_OK;
  if (!ptr_ok(ws)) return OFT_EINVAL;
  return ws_bytes < need ? OFT_EWORKSPACE : OFT_OK;
}

int32_t hip_status(hipError_t e) {
  if (e == hipSuccess) return OFT_OK;
  oft::set_last_hip_error(static_cast<int>(e));
  return OFT_EHIP;
}

}  // namespace

extern "C" {

int32_t oft_vocab_workspace_bytes(const oft_vocab_desc* d, size_t* bytes) {
  if (bytes == nullptr) return OFT_EINVAL;
  const int32_t v = validate_vocab(d);
  if (v != OFT_OK) return v;
  if (d->k < 0 || d->k > OFT_MAX_TEACHER) return OFT_EUNSUPPORTED;
  *bytes = d->T == 0 ? 0 : oft::vocab_ws_bytes(dims(d));
  return OFT_OK;
}

int32_t oft_token_logprobs(const oft_vocab_desc* d, const void* logits, const int32_t* labels_or_null,
                           float* logp_or_null, float* entropy_or_null, int32_t* top_idx_or_null,
                           float* top_logp_or_null, float* stats, void* ws, size_t ws_bytes, void* stream) {
  int32_t v = validate_top(d);
  if (v != OFT_OK) return v;
  if (d->T == 0) return OFT_OK;
  if (!rows_ok(d, logits) || !ptr_ok(stats)) return OFT_EINVAL;
  if ((labels_or_null == nullptr) != (logp_or_null == nullptr)) return OFT_EINVAL;
  if (!opt_ok(labels_or_null) || !opt_ok(logp_or_null) || !opt_ok(entropy_or_null)) return OFT_EINVAL;
  if (d->k > 0 && (!ptr_ok(top_idx_or_null) || !ptr_ok(top_logp_or_null))) return OFT_EINVAL;
  if ((v = ws_ok(d, ws, ws_bytes)) != OFT_OK) return v;
  const oft::LogprobPtrs q{logits,          labels_or_null,   logp_or_null, entropy_or_null,
                           top_idx_or_null, top_logp_or_null, stats};
  return hip_status(
      oft::launch_token_logprobs(dims(d), q, static_cast<char*>(ws), static_cast<hipStream_t>(stream)));
}

int32_t oft_token_logprobs_bwd(const oft_vocab_desc* d, const void* logits, const int32_t* labels_or_null,
                               const float* stats, const float* entropy_or_null, const float* g_logp_or_null,
                               const float* g_entropy_or_null, void* d_logits, void* stream) {
  const int32_t v = validate_vocab(d);
  if (v != OFT_OK) return v;
  if (d->T == 0) return OFT_OK;
  if (!rows_ok(d, logits) || !rows_ok(d, d_logits) || !ptr_ok(stats)) return OFT_EINVAL;
  if ((labels_or_null == nullptr) != (g_logp_or_null == nullptr)) return OFT_EINVAL;
  if (g_logp_or_null == nullptr && g_entropy_or_null == nullptr) return OFT_EINVAL;
  if (g_entropy_or_null != nullptr && entropy_or_null == nullptr) return OFT_EINVAL;
  if (!opt_ok(labels_or_null) || !opt_ok(g_logp_or_null) || !opt_ok(g_entropy_or_null) || !opt_ok(entropy_or_null))
    return OFT_EINVAL;
  if (!grad_rows_ok(d, logits, d_logits)) return OFT_EINVAL;
  const oft::LogprobGradPtrs q{logits,         labels_or_null,    stats,   entropy_or_null,
                               g_logp_or_null, g_entropy_or_null, d_logits};
  return hip_status(oft::launch_token_logprobs_bwd(dims(d), q, static_cast<hipStream_t>(stream)));
}

int32_t oft_distill_topk(const oft_vocab_desc* d, const void* logits, const int32_t* teacher_idx,
                         const float* teacher_logits, float* loss, float* stats, void* ws, size_t ws_bytes,
                         void* stream) {
  int32_t v = validate_teacher(d);
  if (v != OFT_OK) return v;
  if (d->T == 0) return OFT_OK;
  if (!rows_ok(d, logits) || !ptr_ok(teacher_idx) || !ptr_ok(teacher_logits) || !ptr_ok(loss) || !ptr_ok(stats))
    return OFT_EINVAL;
  if ((v = ws_ok(d, ws, ws_bytes)) != OFT_OK) return v;
  return hip_status(oft::launch_distill(dims(d), logits, teacher_idx, teacher_logits, loss, stats,
                                        static_cast<char*>(ws), static_cast<hipStream_t>(stream)));
}

int32_t oft_distill_topk_bwd(const oft_vocab_desc* d, const void* logits, const int32_t* teacher_idx,
                             const float* teacher_logits, const float* stats, const float* g_loss, void* d_logits,
                             void* stream) {
  const int32_t v = validate_teacher(d);
  if (v != OFT_OK) return v;
  if (d->T == 0) return OFT_OK;
  if (!rows_ok(d, logits) || !rows_ok(d, d_logits) || !ptr_ok(teacher_idx) || !ptr_ok(teacher_logits) ||
      !ptr_ok(stats) || !ptr_ok(g_loss))
    return OFT_EINVAL;
  if (!grad_rows_ok(d, logits, d_logits)) return OFT_EINVAL;
  return hip_status(oft::launch_distill_bwd(dims(d), logits, teacher_idx, teacher_logits, stats, g_loss, d_logits,
                                            static_cast<hipStream_t>(stream)));
}

}  // extern "C"
