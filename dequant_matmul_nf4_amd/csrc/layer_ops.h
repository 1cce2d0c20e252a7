// Launches of what stands around the products in a layer and a training step:
// the product with an epilogue, its activation's backward, the routers' balance
// loss, the gradients' norm and clipping.
#pragma once

#include "nf4_internal.h"

struct nf4_grad;

namespace nf4i {

// ---- the product with bias, activation and residual
struct Epilogue {
  const void* bias;          // [rows] float32 or bf16, or null
  int bias_f32;
  int act;                   // nf4_act
  const uint16_t* residual;  // [m][rows] bf16, or null; may be y itself
  uint16_t* pre;             // [m][rows] bf16, or null
};
size_t linear_workspace(int64_t m, int64_t rows, int64_t cols, int r);  // by the sizes alone
hipError_t launch_linear(const uint8_t* packed, int64_t rows, int64_t cols, Scales sc, const uint16_t* x, int64_t m,
                         uint16_t* y, const Epilogue& ep, const uint16_t* lora_a, const uint16_t* lora_b, int r,
                         float lora_scale, void* ws, hipStream_t s);

// ---- dz = dy act'(pre), dbias = its sum over the rows
size_t act_backward_workspace(int64_t m, int64_t rows);
hipError_t launch_act_backward(const uint16_t* dy, const uint16_t* pre, int64_t m, int64_t rows, int act, uint16_t* dz,
                               float* dbias, float* ws, hipStream_t s);

// ---- the routers' balance loss
size_t expert_balance_workspace(int64_t tokens, int experts);
hipError_t launch_expert_balance(const void* logits, int type, const int32_t* ids, const uint8_t* mask, int64_t tokens,
                                 int experts, int slots, float coef, float* loss, int32_t* counts, float* mean_probs,
                                 void* ws, hipStream_t s);
hipError_t launch_expert_balance_backward(const void* logits, int type, const int32_t* counts, const uint8_t* mask,
                                          int64_t tokens, int experts, int slots, float coef, const float* dloss,
                                          void* dlogits, hipStream_t s);

// ---- norm and clipping of many gradients
size_t grad_workspace(int count);
// clip false: the norm alone (the outs are not touched)
hipError_t launch_grads(const nf4_grad* grads, int count, bool clip, float max_norm, const float* total_norm, float* norm,
                        void* ws, hipStream_t s);

}  // namespace nf4i
