// ops_launch.hpp -- host-side launchers of the training and int8 operators
// (internal). Shapes and alignment are validated by the C ABI (ops_api.cpp)
// before any of these runs.
#pragma once

#include "group_launch.hpp"
#include "launch.hpp"

namespace lmhead {

// Softmax cross entropy (xent.hip); arguments already checked.
struct XentForward {
  const void *hidden, *W;  // [M, H], [V, H], both bf16 or both fp16 (in_f16)
  int64_t M, H, V;
  float alpha;
  const float *bias;       // [V] or nullptr
  int in_f16;
  const void *target;      // [M] int64 (target64) or int32
  int target64;
  int64_t ignore;
  float *loss, *lse;       // [M]
  void *workspace;
};
struct XentBackward {
  const void *hidden, *W;
  int64_t M, H, V;
  float alpha;
  const float *bias;
  int in_f16;
  const void *target;
  int target64;
  int64_t ignore;
  const float *lse, *grad_loss;         // [M]
  const float *grad_lse;                // [M] or nullptr
  void *grad_hidden, *grad_W;           // [M, H], [V, H] of the inputs' type; either may be nullptr
  float *grad_bias;                     // [V] or nullptr
  void *workspace;
};
int64_t xent_forward_bytes(int64_t M, int64_t V);
int64_t xent_backward_bytes(int64_t M, int64_t H, int64_t V, bool bias);
hipError_t launch_xent_forward(const XentForward &c, hipStream_t stream);
hipError_t launch_xent_backward(const XentBackward &c, hipStream_t stream);

// Embedding lookup and its gradient (embed.hip); arguments already checked.
struct EmbedForward {
  const void *ids;   // [M] int64 (ids64) or int32
  int ids64;
  int64_t M, H, V;
  const void *W;     // [V, H] bf16, or fp16 (in_f16)
  int in_f16;
  float scale;
  void *out;         // [M, H]
};
struct EmbedBackward {
  const void *ids;
  int ids64;
  int64_t M, H, V;
  const void *grad_out;  // [M, H] bf16, or fp16 (in_f16)
  int in_f16;
  float scale;
  int64_t padding;       // an id without gradient (any value outside [0, V): none)
  int accumulate;
  void *grad_W;          // [V, H]
  void *workspace;
};
int64_t embed_backward_bytes(int64_t M, int64_t H);
hipError_t launch_embed(const EmbedForward &c, hipStream_t stream);
hipError_t launch_embed_backward(const EmbedBackward &c, hipStream_t stream);

// The int8 head (int8.hip); arguments already checked.
struct Int8Args {
  const int8_t *hq;   // [M, H]
  const float *hs;    // [M]
  int64_t M, H;
  const int8_t *wq;   // [V, H]
  const float *ws;    // [V]
  int64_t V;
  float alpha;
  const float *bias;  // [V] or nullptr
  OutType out_type;
  void *out;          // [M, V]
};
hipError_t launch_quantize_int8(const void *x, int64_t rows, int64_t H, int in_f16, int8_t *q, float *scale,
                                hipStream_t stream);
hipError_t launch_int8(const Int8Args &c, hipStream_t stream);

}  // namespace lmhead
