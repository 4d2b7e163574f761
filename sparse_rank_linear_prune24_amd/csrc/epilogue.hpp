// What the fused layer product does between its sums and the store of Y: bias, activation, gate and
// residual in float32, one rounding at the end. Device side of splr_epilogue_t, shared by the
// kernels of every size class.
#pragma once

#include <type_traits>

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

// 1 / (1 + exp(-u)) by the hardware's exp2 and reciprocal (1 ulp each). The rounding of u log2 e is off by
// up to 2^-24 |u| log2 e, which exp turns into a relative error: of u times the result at most 2^-24 u^2
// sigma(u) (1 - sigma(u)), which never exceeds 2^-25 of |u|. Where exp2 overflows the reciprocal is 0,
// the limit.
__device__ __forceinline__ float logistic(float u) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896341f * u));
}

// gelu's Phi(z) as a logistic: log(Phi / (1 - Phi)) = z P(z^2), smooth and odd, so one polynomial serves
// every z without branches. P is a weighted minimax fit on z^2 <= 30 (error of z sigma(z P) at most
// 2.5e-8 |z|); beyond, P stays constant and the logistic goes to 0 or 1 within that error. As evaluated in
// float32 it is 1.6e-7 |z| off at most, the form z (1 + erf(z / sqrt 2)) / 2 with an exact erf 1.0e-7 |z|.
__device__ __forceinline__ float gelu_logit(float z) {
  const float t = fminf(z * z, 30.0f);
  float p = 2.696460242590515e-11f;
  p = fmaf(p, t, 2.342144922451439e-09f);
  p = fmaf(p, t, -2.4576141299803567e-07f);
  p = fmaf(p, t, 7.788853508827742e-06f);
  p = fmaf(p, t, -0.0001100983572541736f);
  p = fmaf(p, t, -6.606032548006624e-05f);
  p = fmaf(p, t, 0.07266674935817719f);
  return z * fmaf(p, t, 1.5957697629928589f);
}

// gelu_tanh is z sigma(2u), the same function as z (1 + tanh u) / 2 without its cancellation.
template <int ACT>
__device__ __forceinline__ f32x4_t activate4(f32x4_t z) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float v = z[e];
    if constexpr (ACT == kActRelu) z[e] = v < 0.0f ? 0.0f : v;
    if constexpr (ACT == kActGelu) z[e] = v * logistic(gelu_logit(v));
    if constexpr (ACT == kActGeluTanh) z[e] = v * logistic(1.5957691216057308f * fmaf(0.044715f * v * v, v, v));
    if constexpr (ACT == kActSilu) z[e] = v * logistic(v);
  }
  return z;
}
// f(std::integral_constant<int, act>{})
template <typename F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    default: f(std::integral_constant<int, kActNone>{}); break;
  }
}
template <typename F>
__device__ __forceinline__ void with_flag(bool flag, F&& f) {
  if (flag) f(std::true_type{});
  else f(std::false_type{});
}

// Four consecutive entries of a float32 or bfloat16 array, as loaded (a bfloat16 quad fills two words):
// those from entry `at` on, of which only the first `left` exist (the others read as 0). vec: all four
// do, aligned to four entries.
__device__ __forceinline__ u32x4_t load_raw4(const void* p, size_t at, bool bf16, bool vec, int left) {
  u32x4_t v = {0, 0, 0, 0};
  if (bf16) {
    const uint16_t* h = (const uint16_t*)p + at;
    if (vec) {
      const u32x2_t w = *(const u32x2_t*)h;
      v[0] = w[0];
      v[1] = w[1];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) v[e / 2] |= (uint32_t)h[e] << (16 * (e & 1));
    }
  } else {
    const uint32_t* f = (const uint32_t*)p + at;
    if (vec) {
      v = *(const u32x4_t*)f;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) v[e] = f[e];
    }
  }
  return v;
}
__device__ __forceinline__ f32x4_t widen4(u32x4_t v, bool bf16) {
  if (!bf16) return __builtin_bit_cast(f32x4_t, v);
  return f32x4_t{__uint_as_float(v[0] << 16), __uint_as_float(v[0] & 0xFFFF0000u), __uint_as_float(v[1] << 16),
                 __uint_as_float(v[1] & 0xFFFF0000u)};
}
__device__ __forceinline__ f32x4_t load4(const void* p, size_t at, bool bf16, bool vec, int left) {
  return widen4(load_raw4(p, at, bf16, vec, left), bf16);
}

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Two float32 values as bfloat16 in one word (hardware conversion, to nearest even; NaN stays NaN)
__device__ __forceinline__ uint32_t round_bf16x2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

template <bool NT>
__device__ __forceinline__ void store4(void* p, size_t at, bool bf16, bool vec, int left, f32x4_t v) {
  if (bf16) {
    uint16_t* h = (uint16_t*)p + at;
    const u32x2_t w = u32x2_t{round_bf16x2(v[0], v[1]), round_bf16x2(v[2], v[3])};
    if (vec) {
      if constexpr (NT) __builtin_nontemporal_store(w, (u32x2_t*)h);
      else *(u32x2_t*)h = w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) h[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
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
  f32x4_t y = sum + bias;
  with_activation(ep.act, [&](auto act) __attribute__((always_inline)) { y = activate4<decltype(act)::value>(y); });
  if (ep.gate) y *= gate;
  if (ep.residual) y += residual;
  return y;
}

}  // namespace
#endif
}  // namespace splr
