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

// 1 / (1 + exp(-u)) in about ten instructions: exp(-u) = 2^h (1 + l ln 2) with h + l = -u log2 e, the
// product carried in two floats so that its rounding is not scaled by |u|; exp2 and reciprocal are the
// hardware's (1 ulp each). Where 2^h overflows, l is dropped and the reciprocal gives 0, the limit.
__device__ __forceinline__ float logistic(float u) {
  constexpr float kLog2e = 1.44269504088896341f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.693147180559945309f;
  const float h = -u * kLog2e;
  const float l = fmaf(-u, kLog2e, -h) - u * kLog2eLow;
  const float p = __builtin_amdgcn_exp2f(h);
  const float e = h > 64.0f ? p : fmaf(p, l * kLn2, p);
  return __builtin_amdgcn_rcpf(1.0f + e);
}

// act on four values; the switch is uniform, so it stays outside the values' code. gelu_tanh is
// z sigma(2u), the same function as z (1 + tanh u) / 2 without its cancellation.
__device__ __forceinline__ f32x4_t activate4(f32x4_t z, int act) {
  switch (act) {
    case kActRelu:
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = z[e] < 0.0f ? 0.0f : z[e];
      break;
    case kActGelu:
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = 0.5f * z[e] * (1.0f + erff(z[e] * 0.70710678118654752f));
      break;
    case kActGeluTanh:
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = 1.5957691216057308f * fmaf(0.044715f * z[e] * z[e], z[e], z[e]);
        z[e] = z[e] * logistic(u);
      }
      break;
    case kActSilu:
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = z[e] * logistic(z[e]);
      break;
    default: break;
  }
  return z;
}

// Four consecutive entries of a float32 or bfloat16 array from entry `at` on, widened; only the first
// `left` exist (the others read as 0). vec: all four do, aligned to four entries.
__device__ __forceinline__ f32x4_t load4(const void* p, size_t at, bool bf16, bool vec, int left) {
  f32x4_t v = {0, 0, 0, 0};
  if (bf16) {
    const uint16_t* h = (const uint16_t*)p + at;
    if (vec) {
      const u32x2_t w = *(const u32x2_t*)h;
      v = f32x4_t{bf16_bits_to_float(w[0] & 0xFFFFu), __uint_as_float(w[0] & 0xFFFF0000u),
                  bf16_bits_to_float(w[1] & 0xFFFFu), __uint_as_float(w[1] & 0xFFFF0000u)};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) v[e] = bf16_bits_to_float(h[e]);
    }
  } else {
    const float* f = (const float*)p + at;
    if (vec) {
      v = *(const f32x4_t*)f;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) v[e] = f[e];
    }
  }
  return v;
}

template <bool NT>
__device__ __forceinline__ void store4(void* p, size_t at, bool bf16, bool vec, int left, f32x4_t v) {
  if (bf16) {
    uint16_t* h = (uint16_t*)p + at;
    uint32_t b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = float_to_bf16_bits(v[e]);
    if (vec) {
      const u32x2_t w = u32x2_t{b[0] | (b[1] << 16), b[2] | (b[3] << 16)};
      if constexpr (NT) __builtin_nontemporal_store(w, (u32x2_t*)h);
      else *(u32x2_t*)h = w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) h[e] = (uint16_t)b[e];
    }
  } else {
    float* f = (float*)p + at;
    if (vec) {
      if constexpr (NT) __builtin_nontemporal_store(v, (f32x4_t*)f);
      else *(f32x4_t*)f = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) f[e] = v[e];
    }
  }
}

// Y's value from the sum, the bias and the gate and residual as loaded
__device__ __forceinline__ f32x4_t finish4(f32x4_t sum, f32x4_t bias, const Epilogue& ep, f32x4_t gate,
                                           f32x4_t residual) {
  f32x4_t y = activate4(sum + bias, ep.act);
  if (ep.gate) y *= gate;
  if (ep.residual) y += residual;
  return y;
}

}  // namespace
#endif
}  // namespace splr
