// losses_launch.hpp -- host-side launchers of the losses over the head's
// logits (losses.hip) and of the rows' top logits (topk.hip); internal. Shapes
// and alignment are validated by the C ABI (losses_api.cpp) before any of these
// runs.
#pragma once

#include "launch.hpp"

namespace lmhead {

// What every loss takes of the head.
struct LossHead {
  const void *hidden, *W;  // [M, H], [V, H], both bf16 or both fp16 (in_f16)
  int64_t M, H, V;
  float alpha;
  const float *bias;       // [V] or nullptr
  float temperature;
  int in_f16;
};
// ... and of memory. state: nullptr when no backward pass follows.
struct LossMemory {
  void *state;
  int keep;                // t is kept in the state (there is one)
  void *workspace;
};
struct LossTargets {
  const void *target;      // [M] int64 (wide) or int32
  int wide;
  int64_t ignore;
};
struct DistillForward {
  LossHead head;
  LossMemory mem;
  const void *ids;         // [M, K] int64 (ids64) or int32
  int ids64;
  int64_t K;
  const void *logits;      // [M, K] of type logits_type
  OutType logits_type;
  const float *teacher_lse;  // [M] or nullptr
  float *loss;             // [M]
};
struct PolicyForward {
  LossHead head;
  LossMemory mem;
  LossTargets y;
  const float *advantage;  // [M]
  const float *old_logp, *ref_logp;  // [M] or nullptr
  float clip_low, clip_high, kl_coef;
  float *loss, *logp;      // [M]
};
struct PreferenceForward {
  LossHead head;
  LossMemory mem;
  LossTargets y;
  const void *starts;      // [2 pairs + 1] int64 (starts64) or int32
  int starts64;
  int64_t pairs;
  const float *ref_logp;   // [2 pairs] or nullptr
  float beta, margin, smoothing;
  int average;
  float *loss, *logp;      // [pairs], [2 pairs]
};
struct LossBackward {
  LossHead head;
  LossMemory mem;          // the state is read
  int64_t K;               // teacher logits a row, 0 for the losses of targets
  const float *grad_loss;
  void *grad_hidden, *grad_W;  // either may be nullptr
  float *grad_bias;            // [V] or nullptr
};
int64_t loss_state_bytes(int64_t M, int64_t H, int64_t V, int64_t K, bool keep);
int64_t loss_forward_bytes(int64_t M, int64_t H, int64_t V, int64_t K, bool with_state);
int64_t loss_backward_bytes(int64_t M, int64_t H, int64_t V, int64_t K, bool keep, bool bias);
hipError_t launch_distill_forward(const DistillForward &c, hipStream_t stream);
hipError_t launch_policy_forward(const PolicyForward &c, hipStream_t stream);
hipError_t launch_preference_forward(const PreferenceForward &c, hipStream_t stream);
hipError_t launch_loss_backward(const LossBackward &c, hipStream_t stream);

struct TopkArgs {
  const void *logits;      // [M, V] of logits_type, rows ld elements apart
  int64_t M, V, ld, K;
  OutType logits_type;
  float temperature;
  void *values;            // [M, K] of logits_type
  int32_t *ids;            // [M, K]
  float *lse;              // [M]
  void *workspace;
};
int64_t topk_bytes(int64_t M, int64_t V, int64_t K);
hipError_t launch_topk(const TopkArgs &c, hipStream_t stream);

}  // namespace lmhead
