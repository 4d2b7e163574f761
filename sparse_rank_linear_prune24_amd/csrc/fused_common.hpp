// Device helpers of the fused products outside the prefill kernel: float32 operands on the bfloat16 matrix
// cores, the rank-r term and the store of accumulator fragments.
//
// In float32 the sparse product runs on the bfloat16 structured-sparse MFMA with float32 accuracy. A float32 number
// has 24 significant bits and a bfloat16 one 8, so x = x1 + x2 + x3 with x1 = RNE(x), x2 = RNE(x - x1),
// x3 = x - x1 - x2, all bfloat16 and the sum exact (|x| from about 1e-30 on; below, x3 may flush). Of the
// nine products of x1 + x2 + x3 and s1 + s2 + s3, each exact in the float32 accumulator, the six of
// order up to 2^-16 are summed; those left out, x2 s3, x3 s2 and x3 s3, are at most 2^-23 of x s (2^-25
// in the mean square), below the rounding of the float32 sum itself. Six structured-sparse MFMAs take
// about 117 cycles for 16 x 16 x 64 where the float32 MFMA needs 512 on an expanded S. An infinite X
// or S entry gives NaN (its low parts are infinity minus infinity).
#pragma once

#include "common.hpp"
#include "epilogue.hpp"

namespace splr {
namespace {

__device__ __forceinline__ f32x4_t mfma_f32(float a, float b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Eight float32 values as three bfloat16 parts (hardware conversion, to nearest even)
struct Parts8 {
  u32x4_t p[3];
};
// four, in two words a part
struct Parts4 {
  u32x2_t p[3];
};
__device__ __forceinline__ Parts4 split3(f32x4_t v) {
  Parts4 o;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f32x2_t x = {v[2 * i], v[2 * i + 1]};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t w = round_bf16x2(x[0], x[1]);
      o.p[k][i] = w;
      x[0] -= __uint_as_float(w << 16);
      x[1] -= __uint_as_float(w & 0xFFFF0000u);
    }
  }
  return o;
}
__device__ __forceinline__ Parts8 split3(f32x4_t lo, f32x4_t hi) {
  const Parts4 l = split3(lo), h = split3(hi);
  Parts8 o;
#pragma unroll
  for (int k = 0; k < 3; ++k) o.p[k] = u32x4_t{l.p[k][0], l.p[k][1], h.p[k][0], h.p[k][1]};
  return o;
}

// acc += S . X^T over one 64-column step, S and X in parts: the small products first
__device__ __forceinline__ f32x4_t product6(const Parts8& s, const bf16x16_t (&x)[3], int idx, f32x4_t acc) {
  acc = smfmac16x16x64(as_bf16x8(s.p[2]), x[0], acc, idx);
  acc = smfmac16x16x64(as_bf16x8(s.p[0]), x[2], acc, idx);
  acc = smfmac16x16x64(as_bf16x8(s.p[1]), x[1], acc, idx);
  acc = smfmac16x16x64(as_bf16x8(s.p[1]), x[0], acc, idx);
  acc = smfmac16x16x64(as_bf16x8(s.p[0]), x[1], acc, idx);
  return smfmac16x16x64(as_bf16x8(s.p[0]), x[0], acc, idx);
}

// Finishes and stores acc[i][j]: rows n0 + 16 i + 4 quad .. +3, token m0 + 16 j + sub (of the rows from
// row0 on)
template <int NI, int NJ>
__device__ __forceinline__ void store_fragments(const f32x4_t (&acc)[NI][NJ], const Epilogue& ep, size_t bias_row,
                                                void* Y, int y_bf16, int M, int n_out, int n0, int m0, size_t row0,
                                                int sub, int quad) {
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int n = n0 + 16 * i + 4 * quad, left = n_out - n;
    if (left <= 0) continue;
    const bool vec = (n_out & 3) == 0 && left >= 4;
    f32x4_t bias = {0, 0, 0, 0}, gate[NJ], residual[NJ];
    if (ep.bias) bias = load4(ep.bias, bias_row + n, ep.bias_bf16, vec, left);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const size_t at = (row0 + min(m0 + 16 * j + sub, M - 1)) * n_out + n;
      if (ep.gate) gate[j] = load4(ep.gate, at, y_bf16, vec, left);
      if (ep.residual) residual[j] = load4(ep.residual, at, y_bf16, vec, left);
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int m = m0 + 16 * j + sub;
      const f32x4_t y = finish4(acc[i][j], bias, ep, gate[j], residual[j]);
      if (m < M) store4<false>(Y, (row0 + m) * n_out + n, y_bf16, vec, left, y);
    }
  }
}

}  // namespace
}  // namespace splr
