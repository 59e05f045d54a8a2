// ops_api.cpp -- the C ABI of the training and int8 operators: argument checks
// and launch. As in lmhead_api.cpp, every check is host-side integer work done
// before anything is enqueued; a call that fails one launches nothing.
#include "../../include/lmhead.h"

#include <hip/hip_runtime.h>

#include "ops_launch.hpp"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool known_dtype(int d) { return d == LMHEAD_F32 || d == LMHEAD_BF16 || d == LMHEAD_F16; }

// The shape contract of the projection (its M * V bound included).
lmhead_status check_shape(int64_t M, int64_t H, int64_t V) {
  if (M < 0 || H <= 0 || V <= 0) return LMHEAD_ERR_INVALID;
  if (M > LMHEAD_MAX_M || H > LMHEAD_MAX_H || V > LMHEAD_MAX_V) return LMHEAD_ERR_INVALID;
  if (M > 0 && M > ((int64_t)1 << 42) / V) return LMHEAD_ERR_INVALID;
  return H % 32 != 0 ? LMHEAD_NOT_HANDLED : LMHEAD_OK;
}

// ... and 16-bit tensors of type `dtype`.
lmhead_status check_call(int64_t M, int64_t H, int64_t V, int dtype) {
  const lmhead_status st = check_shape(M, H, V);
  if (st != LMHEAD_OK) return st;
  if (!known_dtype(dtype)) return LMHEAD_ERR_INVALID;
  return dtype == LMHEAD_F32 ? LMHEAD_NOT_HANDLED : LMHEAD_OK;
}

}  // namespace

extern "C" {

size_t lmhead_xent_forward_workspace_bytes(int64_t M, int64_t V) {
  if (check_shape(M, 32, V) == LMHEAD_ERR_INVALID) return 0;
  return (size_t)lmhead::xent_forward_bytes(M, V);
}

size_t lmhead_xent_backward_workspace_bytes(int64_t M, int64_t H, int64_t V, int grad_bias) {
  if (check_shape(M, H, V) != LMHEAD_OK || M == 0) return 0;
  return (size_t)lmhead::xent_backward_bytes(M, H, V, grad_bias != 0);
}

lmhead_status lmhead_xent_forward(const void *hidden, int64_t M, int64_t H, const void *W, int64_t V,
                                  float alpha, const float *bias, lmhead_dtype in_dtype,
                                  const void *target, lmhead_index target_type,
                                  int64_t ignore_index, float *loss, float *lse, void *workspace,
                                  size_t workspace_bytes, void *stream) {
  lmhead_status st = check_call(M, H, V, in_dtype);
  if (st != LMHEAD_OK) return st;
  if (target_type != LMHEAD_INDEX32 && target_type != LMHEAD_INDEX64) return LMHEAD_ERR_INVALID;
  if (M == 0) return LMHEAD_OK;
  if (hidden == nullptr || W == nullptr || target == nullptr || loss == nullptr || lse == nullptr ||
      workspace == nullptr || workspace_bytes < lmhead_xent_forward_workspace_bytes(M, V))
    return LMHEAD_ERR_INVALID;
  if (!aligned(hidden, 16) || !aligned(W, 16) || !aligned(target, target_type == LMHEAD_INDEX64 ? 8 : 4) ||
      !aligned(loss, 4) || !aligned(lse, 4) || !aligned(bias, 4) || !aligned(workspace, 16))
    return LMHEAD_ERR_ALIGN;
  const lmhead::XentForward c{hidden, W, M, H, V, alpha, bias, in_dtype == LMHEAD_F16 ? 1 : 0, target,
                              target_type == LMHEAD_INDEX64 ? 1 : 0, ignore_index, loss, lse, workspace};
  hipError_t e = lmhead::launch_xent_forward(c, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? LMHEAD_OK : LMHEAD_ERR_DEVICE;
}

lmhead_status lmhead_xent_backward(const void *hidden, int64_t M, int64_t H, const void *W, int64_t V,
                                   float alpha, const float *bias, lmhead_dtype in_dtype,
                                   const void *target, lmhead_index target_type,
                                   int64_t ignore_index, const float *lse, const float *grad_loss,
                                   const float *grad_lse, void *grad_hidden, void *grad_W,
                                   float *grad_bias, void *workspace, size_t workspace_bytes,
                                   void *stream) {
  lmhead_status st = check_call(M, H, V, in_dtype);
  if (st != LMHEAD_OK) return st;
  if (target_type != LMHEAD_INDEX32 && target_type != LMHEAD_INDEX64) return LMHEAD_ERR_INVALID;
  if (grad_hidden == nullptr && grad_W == nullptr && grad_bias == nullptr) return LMHEAD_OK;
  if (M > 0) {
    if (hidden == nullptr || W == nullptr || target == nullptr || lse == nullptr || grad_loss == nullptr ||
        workspace == nullptr ||
        workspace_bytes < lmhead_xent_backward_workspace_bytes(M, H, V, grad_bias != nullptr))
      return LMHEAD_ERR_INVALID;
    if (!aligned(hidden, 16) || !aligned(W, 16) ||
        !aligned(target, target_type == LMHEAD_INDEX64 ? 8 : 4) || !aligned(lse, 4) ||
        !aligned(grad_loss, 4) || !aligned(grad_lse, 4) || !aligned(bias, 4) || !aligned(workspace, 256))
      return LMHEAD_ERR_ALIGN;
  }
  if (!aligned(grad_hidden, 16) || !aligned(grad_W, 16) || !aligned(grad_bias, 4)) return LMHEAD_ERR_ALIGN;
  const lmhead::XentBackward c{hidden, W, M, H, V, alpha, bias, in_dtype == LMHEAD_F16 ? 1 : 0, target,
                               target_type == LMHEAD_INDEX64 ? 1 : 0, ignore_index, lse, grad_loss,
                               grad_lse, grad_hidden, grad_W, grad_bias, workspace};
  hipError_t e = lmhead::launch_xent_backward(c, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? LMHEAD_OK : LMHEAD_ERR_DEVICE;
}

lmhead_status lmhead_embed(const void *ids, lmhead_index ids_type, int64_t M, const void *W, int64_t V,
                           int64_t H, lmhead_dtype dtype, float scale, void *out, void *stream) {
  lmhead_status st = check_call(M, H, V, dtype);
  if (st != LMHEAD_OK) return st;
  if (ids_type != LMHEAD_INDEX32 && ids_type != LMHEAD_INDEX64) return LMHEAD_ERR_INVALID;
  if (M == 0) return LMHEAD_OK;
  if (ids == nullptr || W == nullptr || out == nullptr) return LMHEAD_ERR_INVALID;
  if (!aligned(ids, ids_type == LMHEAD_INDEX64 ? 8 : 4) || !aligned(W, 16) || !aligned(out, 16))
    return LMHEAD_ERR_ALIGN;
  const lmhead::EmbedForward c{ids, ids_type == LMHEAD_INDEX64 ? 1 : 0, M, H, V, W,
                               dtype == LMHEAD_F16 ? 1 : 0, scale, out};
  hipError_t e = lmhead::launch_embed(c, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? LMHEAD_OK : LMHEAD_ERR_DEVICE;
}

size_t lmhead_embed_backward_workspace_bytes(int64_t M, int64_t H) {
  if (check_shape(M, H, 1) != LMHEAD_OK) return 0;
  return (size_t)lmhead::embed_backward_bytes(M, H);
}

lmhead_status lmhead_embed_backward(const void *ids, lmhead_index ids_type, int64_t M, const void *grad_out,
                                    int64_t V, int64_t H, lmhead_dtype dtype, float scale,
                                    int64_t padding_index, int accumulate, void *grad_W, void *workspace,
                                    size_t workspace_bytes, void *stream) {
  lmhead_status st = check_call(M, H, V, dtype);
  if (st != LMHEAD_OK) return st;
  if (ids_type != LMHEAD_INDEX32 && ids_type != LMHEAD_INDEX64) return LMHEAD_ERR_INVALID;
  if (grad_W == nullptr) return LMHEAD_ERR_INVALID;
  if (M > 0 && (ids == nullptr || grad_out == nullptr || workspace == nullptr ||
                workspace_bytes < lmhead_embed_backward_workspace_bytes(M, H)))
    return LMHEAD_ERR_INVALID;
  if (!aligned(grad_W, 16)) return LMHEAD_ERR_ALIGN;
  if (M > 0 && (!aligned(ids, ids_type == LMHEAD_INDEX64 ? 8 : 4) || !aligned(grad_out, 16) ||
                !aligned(workspace, 256)))
    return LMHEAD_ERR_ALIGN;
  const lmhead::EmbedBackward c{ids, ids_type == LMHEAD_INDEX64 ? 1 : 0, M, H, V, grad_out,
                                dtype == LMHEAD_F16 ? 1 : 0, scale, padding_index, accumulate != 0, grad_W,
                                workspace};
  hipError_t e = lmhead::launch_embed_backward(c, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? LMHEAD_OK : LMHEAD_ERR_DEVICE;
}

lmhead_status lmhead_quantize_int8(const void *x, int64_t rows, int64_t H, lmhead_dtype dtype, int8_t *codes,
                                   float *scales, void *stream) {
  lmhead_status st = check_call(rows, H, 1, dtype);
  if (st != LMHEAD_OK || rows == 0) return st;
  if (x == nullptr || codes == nullptr || scales == nullptr) return LMHEAD_ERR_INVALID;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return LMHEAD_ERR_ALIGN;
  hipError_t e = lmhead::launch_quantize_int8(x, rows, H, dtype == LMHEAD_F16 ? 1 : 0, codes, scales,
                                              static_cast<hipStream_t>(stream));
  return e == hipSuccess ? LMHEAD_OK : LMHEAD_ERR_DEVICE;
}

lmhead_status lmhead_logits_int8(const int8_t *hidden, const float *hidden_scale, int64_t M, int64_t H,
                                 const int8_t *W, const float *w_scale, int64_t V, float alpha,
                                 const float *bias, lmhead_dtype out_dtype, void *out, void *stream) {
  lmhead_status st = check_shape(M, H, V);
  if (st != LMHEAD_OK) return st;
  if (!known_dtype(out_dtype)) return LMHEAD_ERR_INVALID;
  if (M == 0) return LMHEAD_OK;
  if (hidden == nullptr || hidden_scale == nullptr || W == nullptr || w_scale == nullptr || out == nullptr)
    return LMHEAD_ERR_INVALID;
  if (!aligned(hidden, 16) || !aligned(W, 16) || !aligned(out, 16) || !aligned(hidden_scale, 4) ||
      !aligned(w_scale, 4) || !aligned(bias, 4))
    return LMHEAD_ERR_ALIGN;
  const lmhead::Int8Args c{hidden, hidden_scale, M, H, W, w_scale, V, alpha, bias,
                           out_dtype == LMHEAD_F32    ? lmhead::OUT_F32
                           : out_dtype == LMHEAD_BF16 ? lmhead::OUT_BF16
                                                      : lmhead::OUT_F16,
                           out};
  hipError_t e = lmhead::launch_int8(c, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? LMHEAD_OK : LMHEAD_ERR_DEVICE;
}

}  // extern "C"
