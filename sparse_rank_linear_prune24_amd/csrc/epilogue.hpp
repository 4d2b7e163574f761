// What the fused layer product does between its sums and the store of Y: bias, activation, gate and
// residual in float32, one rounding at the end. Device side of splr_epilogue_t, shared by the
// kernels of every size class.
#pragma once

#include "common.hpp"

namespace splr {

// Operands as the kernels take them (a NULL one is left out). bias is float32 or bfloat16 as the
// call's dtype, gate and residual as Y.
struct Epilogue {
  const void* bias;
  const void* gate;
  const void* residual;
  int act;        // splr_activation_t
  int bias_bf16;
};
enum : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4, kActCount = 5 };

#ifdef __HIPCC__
namespace {

__device__ __forceinline__ float load_as_float(const void* p, size_t i, bool bf16) {
  return bf16 ? bf16_bits_to_float(((const uint16_t*)p)[i]) : ((const float*)p)[i];
}

// The logistic forms divide by 1 + exp(-u): where exp overflows the quotient is -0, the limit.
// gelu_tanh is z sigma(2u), the same function as z (1 + tanh u) / 2 without its cancellation.
__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case kActRelu: return z < 0.0f ? 0.0f : z;
    case kActGelu: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case kActGeluTanh: return z / (1.0f + expf(-1.5957691216057308f * (z + 0.044715f * z * z * z)));
    case kActSilu: return z / (1.0f + expf(-z));
    default: return z;
  }
}

}  // namespace
#endif
}  // namespace splr
