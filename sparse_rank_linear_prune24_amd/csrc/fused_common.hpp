// Device helpers of the fused products outside the prefill kernel: float32 operands on the bfloat16 matrix
// cores, the rank-r term and the store of accumulator fragments.
//
// In float32 the sparse product runs on the bfloat16 structured-sparse MFMA with float32 accuracy. A float32 number
// has 24 significant bits and a bfloat16 one 8, so x = x1 + x2 + x3 with x1 = RNE(x), x2 = RNE(x - x1),
// x3 = x - x1 - x2, all bfloat16 and the sum exact (|x| from 2^-110 on; below, x3 is rounded to a multiple
// of 2^-133, bfloat16's least number, which the conversions and the MFMA keep). Of the
// nine products of x1 + x2 + x3 and s1 + s2 + s3, each exact in the float32 accumulator, the six of
// order up to 2^-16 are summed; those left out, x2 s3, x3 s2 and x3 s3, are at most 2^-23 of x s (2^-25
// in the mean square), below the rounding of the float32 sum itself. Six structured-sparse MFMAs take
// about 117 cycles for 16 x 16 x 64 where the float32 MFMA needs 512 on an expanded S. An infinite X or S
// entry, or one above 3.39e38 (x1 rounds to infinity), makes its sums NaN, since the low parts are infinity
// minus infinity: sums that end as NaN are formed once more, in float32 (resum_nan).
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

// Row `row` of a tile row of S (its values and metadata from their first tile column on) times x, over the kept
// entries in order; NaN as soon as the sum is (K is a multiple of 32, so of the 16 columns of a round)
__device__ __forceinline__ float sparse_dot(const float* __restrict__ x, const float* __restrict__ values,
                                            const uint32_t* __restrict__ meta, int row, int K) {
  float sum = 0.0f;
  for (int g0 = 0; g0 < K / 4 && sum == sum; g0 += 4) {
    const int tk = g0 / 16, lane = row + 16 * (g0 % 16 / 4);
    const uint32_t unit = meta_unit(meta, 0, 0, tk, lane);
    const float* kept = values + (size_t)tk * 512 + lane * 8;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint32_t nib = unit >> (4 * g);
      sum = fmaf(x[4 * (g0 + g) + (nib & 3u)], kept[2 * g], sum);
      sum = fmaf(x[4 * (g0 + g) + ((nib >> 2) & 3u)], kept[2 * g + 1], sum);
    }
  }
  return sum;
}

// Forms those of the sums acc[i][j] that are NaN again, so that operands which the bfloat16 parts cannot carry give
// what float32 gives. Layout as store_fragments; values and meta: S of the tile row of n0, TK and TKB its
// blocks a tile row. Without such sums this is half a comparison for each (0 to 0.3 us a call). With them the
// wave walks K for each, until the sum is NaN again if it is: 1000 rows 2048 -> 2050 take 68 us, with one infinite
// entry 590, with a row of NaN 67 and with NaN everywhere 111 (the plain float32 product 780).
template <int NI, int NJ>
__device__ __forceinline__ void resum_nan(f32x4_t (&acc)[NI][NJ], const float* __restrict__ X,
                                          const float* __restrict__ values, const uint32_t* __restrict__ meta, int K,
                                          int M, int n_out, int n0, int m0, int sub, int quad) {
  const auto any_nan = [](f32x4_t v) { return __builtin_isunordered(v[0], v[1]) || __builtin_isunordered(v[2], v[3]); };
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) nan |= any_nan(acc[i][j]);
  if (__builtin_expect(!__any(nan), 1)) return;
  const int TK = (K + 63) / 64, TKB = meta_blocks(TK);
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int m = m0 + 16 * j + sub, n = n0 + 16 * i + 4 * quad;
      const f32x4_t v = acc[i][j];
      if (!any_nan(v)) continue;
#pragma unroll 1
      for (int e = 0; e < 4; ++e) {
        const float old = e == 0 ? v[0] : e == 1 ? v[1] : e == 2 ? v[2] : v[3];
        if (old == old || m >= M || n + e >= n_out) continue;
        const float sum = sparse_dot(X + (size_t)m * K, values + (size_t)i * TK * 512, meta + (size_t)i * TKB * 256,
                                     4 * quad + e, K);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][j][k] = e == k ? sum : acc[i][j][k];
      }
    }
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
