// losses_api.cpp -- the C ABI of the losses over the head's logits and of the
// rows' top logits: argument checks and launch. As in lmhead_api.cpp, every
// check is host-side work done before anything is enqueued; a call that fails
// one launches nothing.
#include "../../include/lmhead.h"

#include <hip/hip_runtime.h>
#include <math.h>

#include "losses_launch.hpp"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool known_dtype(int d) { return d == LMHEAD_F32 || d == LMHEAD_BF16 || d == LMHEAD_F16; }
bool known_index(int t) { return t == LMHEAD_INDEX32 || t == LMHEAD_INDEX64; }
uintptr_t index_size(int t) { return t == LMHEAD_INDEX64 ? 8 : 4; }

// The shape contract of the projection (its M * V bound included).
lmhead_status check_shape(int64_t M, int64_t H, int64_t V) {
  if (M < 0 || H <= 0 || V <= 0) return LMHEAD_ERR_INVALID;
  if (M > LMHEAD_MAX_M || H > LMHEAD_MAX_H || V > LMHEAD_MAX_V) return LMHEAD_ERR_INVALID;
  if (M > 0 && M > ((int64_t)1 << 42) / V) return LMHEAD_ERR_INVALID;
  return H % 32 != 0 ? LMHEAD_NOT_HANDLED : LMHEAD_OK;
}

// ... 16-bit tensors of type `dtype`, and a temperature that divides.
lmhead_status check_head(int64_t M, int64_t H, int64_t V, int dtype, float temperature) {
  const lmhead_status st = check_shape(M, H, V);
  if (st != LMHEAD_OK) return st;
  if (!known_dtype(dtype) || !(temperature > 0.0f) || isinf(temperature)) return LMHEAD_ERR_INVALID;
  return dtype == LMHEAD_F32 ? LMHEAD_NOT_HANDLED : LMHEAD_OK;
}

lmhead::LossHead head_of(const void *hidden, int64_t M, int64_t H, const void *W, int64_t V, float alpha,
                         const float *bias, int dtype, float temperature) {
  return lmhead::LossHead{hidden, W, M, H, V, alpha, bias, temperature, dtype == LMHEAD_F16 ? 1 : 0};
}

// The memory of a forward pass over M > 0 rows.
lmhead_status check_forward(const lmhead::LossHead &h, int64_t K, const void *state, size_t state_bytes,
                            int keep_logits, const void *workspace, size_t workspace_bytes) {
  if (h.hidden == nullptr || h.W == nullptr || workspace == nullptr ||
      workspace_bytes < (size_t)lmhead::loss_forward_bytes(h.M, h.H, h.V, K, state != nullptr) ||
      (state != nullptr && state_bytes < (size_t)lmhead::loss_state_bytes(h.M, h.H, h.V, K, keep_logits != 0)) ||
      (state == nullptr && keep_logits != 0))
    return LMHEAD_ERR_INVALID;
  if (!aligned(h.hidden, 16) || !aligned(h.W, 16) || !aligned(h.bias, 4) || !aligned(state, 256) ||
      !aligned(workspace, 256))
    return LMHEAD_ERR_ALIGN;
  return LMHEAD_OK;
}

bool teacher_count_ok(int64_t K) { return K >= 0 && K <= LMHEAD_MAX_TEACHER; }

lmhead::OutType out_type(int dtype) {
  return dtype == LMHEAD_F32 ? lmhead::OUT_F32 : dtype == LMHEAD_BF16 ? lmhead::OUT_BF16 : lmhead::OUT_F16;
}

lmhead_status done(hipError_t e) { return e == hipSuccess ? LMHEAD_OK : LMHEAD_ERR_DEVICE; }

}  // namespace

extern "C" {

size_t lmhead_logits_topk_workspace_bytes(int64_t M, int64_t V, int64_t K) {
  if (check_shape(M, 32, V) != LMHEAD_OK || M == 0 || K < 1 || K > LMHEAD_MAX_TOPK || K > V) return 0;
  return (size_t)lmhead::topk_bytes(M, V, K);
}

lmhead_status lmhead_logits_topk(const void *logits, int64_t M, int64_t V, int64_t row_stride, lmhead_dtype dtype, int64_t K,
                                 float temperature, void *values, int32_t *ids, float *lse, void *workspace,
                                 size_t workspace_bytes, void *stream) {
  const lmhead_status st = check_shape(M, 32, V);
  if (st != LMHEAD_OK) return st;
  if (!known_dtype(dtype) || K < 1 || K > LMHEAD_MAX_TOPK || K > V || row_stride < V || row_stride > (int64_t)1 << 40 ||
      !(temperature > 0.0f) || isinf(temperature))
    return LMHEAD_ERR_INVALID;
  if (M == 0) return LMHEAD_OK;
  const size_t need = lmhead_logits_topk_workspace_bytes(M, V, K);
  if (logits == nullptr || values == nullptr || ids == nullptr || lse == nullptr ||
      (need > 0 && (workspace == nullptr || workspace_bytes < need)))
    return LMHEAD_ERR_INVALID;
  const uintptr_t size = dtype == LMHEAD_F32 ? 4 : 2;
  if (!aligned(logits, size) || !aligned(values, size) || !aligned(ids, 4) || !aligned(lse, 4) || !aligned(workspace, 16))
    return LMHEAD_ERR_ALIGN;
  return done(lmhead::launch_topk(lmhead::TopkArgs{logits, M, V, row_stride, K, out_type(dtype), temperature, values, ids,
                                                   lse, workspace},
                                  static_cast<hipStream_t>(stream)));
}

size_t lmhead_loss_state_bytes(int64_t M, int64_t H, int64_t V, int64_t K, int keep_logits) {
  if (check_shape(M, H, V) != LMHEAD_OK || M == 0 || !teacher_count_ok(K)) return 0;
  return (size_t)lmhead::loss_state_bytes(M, H, V, K, keep_logits != 0);
}

size_t lmhead_loss_forward_workspace_bytes(int64_t M, int64_t H, int64_t V, int64_t K, int with_state) {
  if (check_shape(M, H, V) != LMHEAD_OK || M == 0 || !teacher_count_ok(K)) return 0;
  return (size_t)lmhead::loss_forward_bytes(M, H, V, K, with_state != 0);
}

size_t lmhead_loss_backward_workspace_bytes(int64_t M, int64_t H, int64_t V, int64_t K, int keep_logits,
                                            int grad_bias) {
  if (check_shape(M, H, V) != LMHEAD_OK || M == 0 || !teacher_count_ok(K)) return 0;
  return (size_t)lmhead::loss_backward_bytes(M, H, V, K, keep_logits != 0, grad_bias != 0);
}

lmhead_status lmhead_distill_forward(const void *hidden, int64_t M, int64_t H, const void *W, int64_t V, float alpha,
                                     const float *bias, lmhead_dtype in_dtype, float temperature,
                                     const void *teacher_ids, lmhead_index ids_type, const void *teacher_logits,
                                     lmhead_dtype logits_dtype, int64_t K, const float *teacher_lse, float *loss,
                                     void *state, size_t state_bytes, int keep_logits, void *workspace, size_t workspace_bytes,
                                     void *stream) {
  lmhead_status st = check_head(M, H, V, in_dtype, temperature);
  if (st != LMHEAD_OK) return st;
  if (!known_index(ids_type) || !known_dtype(logits_dtype) || K < 1 || !teacher_count_ok(K)) return LMHEAD_ERR_INVALID;
  if (M == 0) return LMHEAD_OK;
  const lmhead::LossHead h = head_of(hidden, M, H, W, V, alpha, bias, in_dtype, temperature);
  st = check_forward(h, K, state, state_bytes, keep_logits, workspace, workspace_bytes);
  if (st == LMHEAD_ERR_INVALID || teacher_ids == nullptr || teacher_logits == nullptr || loss == nullptr)
    return LMHEAD_ERR_INVALID;
  if (st != LMHEAD_OK || !aligned(teacher_ids, index_size(ids_type)) ||
      !aligned(teacher_logits, logits_dtype == LMHEAD_F32 ? 4 : 2) || !aligned(teacher_lse, 4) || !aligned(loss, 4))
    return LMHEAD_ERR_ALIGN;
  return done(lmhead::launch_distill_forward(
      lmhead::DistillForward{h, lmhead::LossMemory{state, keep_logits != 0, workspace}, teacher_ids, ids_type == LMHEAD_INDEX64 ? 1 : 0, K,
                             teacher_logits,
                             out_type(logits_dtype), teacher_lse, loss},
      static_cast<hipStream_t>(stream)));
}

lmhead_status lmhead_policy_forward(const void *hidden, int64_t M, int64_t H, const void *W, int64_t V, float alpha,
                                    const float *bias, lmhead_dtype in_dtype, float temperature, const void *target,
                                    lmhead_index target_type, int64_t ignore_index, const float *advantage,
                                    const float *old_logp, const float *ref_logp, float clip_low, float clip_high,
                                    float kl_coef, float *loss, float *logp, void *state, size_t state_bytes, int keep_logits,
                                    void *workspace, size_t workspace_bytes, void *stream) {
  lmhead_status st = check_head(M, H, V, in_dtype, temperature);
  if (st != LMHEAD_OK) return st;
  if (!known_index(target_type) || !(clip_low >= 0.0f) || !(clip_high >= 0.0f) || kl_coef != kl_coef)
    return LMHEAD_ERR_INVALID;
  if (M == 0) return LMHEAD_OK;
  const lmhead::LossHead h = head_of(hidden, M, H, W, V, alpha, bias, in_dtype, temperature);
  st = check_forward(h, 0, state, state_bytes, keep_logits, workspace, workspace_bytes);
  if (st == LMHEAD_ERR_INVALID || target == nullptr || advantage == nullptr || loss == nullptr || logp == nullptr)
    return LMHEAD_ERR_INVALID;
  if (st != LMHEAD_OK || !aligned(target, index_size(target_type)) || !aligned(advantage, 4) || !aligned(old_logp, 4) ||
      !aligned(ref_logp, 4) || !aligned(loss, 4) || !aligned(logp, 4))
    return LMHEAD_ERR_ALIGN;
  return done(lmhead::launch_policy_forward(
      lmhead::PolicyForward{h, lmhead::LossMemory{state, keep_logits != 0, workspace},
                            lmhead::LossTargets{target, target_type == LMHEAD_INDEX64 ? 1 : 0, ignore_index}, advantage,
                            old_logp, ref_logp, clip_low, clip_high, kl_coef, loss, logp},
      static_cast<hipStream_t>(stream)));
}

lmhead_status lmhead_preference_forward(const void *hidden, int64_t M, int64_t H, const void *W, int64_t V, float alpha,
                                        const float *bias, lmhead_dtype in_dtype, float temperature, const void *target,
                                        lmhead_index target_type, int64_t ignore_index, const void *starts,
                                        lmhead_index starts_type, int64_t pairs, const float *ref_logp, float beta,
                                        float margin, float label_smoothing, int average, float *loss, float *logp,
                                        void *state, size_t state_bytes, int keep_logits, void *workspace, size_t workspace_bytes,
                                        void *stream) {
  lmhead_status st = check_head(M, H, V, in_dtype, temperature);
  if (st != LMHEAD_OK) return st;
  if (!known_index(target_type) || !known_index(starts_type) || pairs < 0 || pairs > LMHEAD_MAX_M / 2 ||
      !(label_smoothing >= 0.0f && label_smoothing <= 1.0f) || beta != beta || margin != margin)
    return LMHEAD_ERR_INVALID;
  const lmhead::LossHead h = head_of(hidden, M, H, W, V, alpha, bias, in_dtype, temperature);
  if (pairs > 0 && (starts == nullptr || loss == nullptr || logp == nullptr)) return LMHEAD_ERR_INVALID;
  if (M > 0) {
    if (target == nullptr) return LMHEAD_ERR_INVALID;
    st = check_forward(h, 0, state, state_bytes, keep_logits, workspace, workspace_bytes);
    if (st != LMHEAD_OK) return st;
  }
  if (!aligned(target, index_size(target_type)) || !aligned(starts, index_size(starts_type)) || !aligned(ref_logp, 4) ||
      !aligned(loss, 4) || !aligned(logp, 4))
    return LMHEAD_ERR_ALIGN;
  return done(lmhead::launch_preference_forward(
      lmhead::PreferenceForward{h, lmhead::LossMemory{state, keep_logits != 0, workspace},
                                lmhead::LossTargets{target, target_type == LMHEAD_INDEX64 ? 1 : 0, ignore_index}, starts,
                                starts_type == LMHEAD_INDEX64 ? 1 : 0, pairs, ref_logp, beta, margin, label_smoothing,
                                average != 0, loss, logp},
      static_cast<hipStream_t>(stream)));
}

lmhead_status lmhead_loss_backward(const void *hidden, int64_t M, int64_t H, const void *W, int64_t V, float alpha,
                                   const float *bias, lmhead_dtype in_dtype, float temperature, int64_t K,
                                   const float *grad_loss, const void *state, size_t state_bytes, int keep_logits, void *grad_hidden,
                                   void *grad_W, float *grad_bias, void *workspace, size_t workspace_bytes,
                                   void *stream) {
  lmhead_status st = check_head(M, H, V, in_dtype, temperature);
  if (st != LMHEAD_OK) return st;
  if (!teacher_count_ok(K)) return LMHEAD_ERR_INVALID;
  if (grad_hidden == nullptr && grad_W == nullptr && grad_bias == nullptr) return LMHEAD_OK;
  if (M > 0) {
    if (hidden == nullptr || W == nullptr || state == nullptr ||
        state_bytes < lmhead_loss_state_bytes(M, H, V, K, keep_logits) || workspace == nullptr ||
        workspace_bytes < lmhead_loss_backward_workspace_bytes(M, H, V, K, keep_logits, grad_bias != nullptr))
      return LMHEAD_ERR_INVALID;
    if (!aligned(hidden, 16) || !aligned(W, 16) || !aligned(bias, 4) || !aligned(grad_loss, 4) || !aligned(state, 256) ||
        !aligned(workspace, 256))
      return LMHEAD_ERR_ALIGN;
  }
  if (!aligned(grad_hidden, 16) || !aligned(grad_W, 16) || !aligned(grad_bias, 4)) return LMHEAD_ERR_ALIGN;
  return done(lmhead::launch_loss_backward(
      lmhead::LossBackward{head_of(hidden, M, H, W, V, alpha, bias, in_dtype, temperature),
                           lmhead::LossMemory{const_cast<void *>(state), keep_logits != 0, workspace}, K, grad_loss, grad_hidden, grad_W,
                           grad_bias},
      static_cast<hipStream_t>(stream)));
}

}  // extern "C"
