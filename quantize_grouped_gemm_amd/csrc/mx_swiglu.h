// SwiGLU's gradient, shared by the kernels that take its input in bf16
// (mx_quant.hip) and from the 8-bit checkpoint (mx_swiglu_ck.hip). The forward
// (swiglu_pair) is in mx_tile.h.
#pragma once

#include "mx_tile.h"

namespace mxk {

// dA = dh*b*s*(1 + a*(1-s)), dB = dh*a*s with s = sigmoid(a), float32.
__device__ __forceinline__ void swiglu_grad_f32(float dh, float a, float b, float& da,
                                                float& db) {
  const float s = sigmoid_f32(a);
  da = (dh * b) * (s * (1.0f + a * (1.0f - s)));
  db = dh * (a * s);
}

__device__ __forceinline__ void swiglu_grad_pair(uint32_t wdh, uint32_t wa, uint32_t wb,
                                                 uint32_t& da2, uint32_t& db2) {
  float da0, db0, da1, db1;
  swiglu_grad_f32(bf16_lo(wdh), bf16_lo(wa), bf16_lo(wb), da0, db0);
  swiglu_grad_f32(bf16_hi(wdh), bf16_hi(wa), bf16_hi(wb), da1, db1);
  da2 = pack_bf16x2(da0, da1);
  db2 = pack_bf16x2(db0, db1);
}

}  // namespace mxk
