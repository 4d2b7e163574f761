// Entries in 8 bits (e4m3: 4 exponent bits, 3 mantissa bits, largest 448, no infinities, NaN 0x7F or 0xFF) with a float32 scale for
// each block: device helpers of the quantisation and of the products that read it, and what a product call holds.
#pragma once

#include "common.hpp"
#include "epilogue.hpp"
#include "groups.hpp"
#include "kernels.hpp"

namespace splr {

constexpr int kBlockK = 128;  // entries of a block along the reduction dimension

// A call's operands, as its launchers take them.
struct Fp8Call {
  const void* X;          // [M][n_in]
  int x_type;             // splr_dtype_t: e4m3, or what the call quantises
  const float* x_scales;  // [ceil(n_in / 128)][M]
  int64_t M, n_in;
  const int32_t* offsets;  // NULL: one layer
  int64_t experts;
  const uint8_t* W;       // [experts][n_out][n_in]
  const float* w_scales;  // blocks of 128 rows: [ceil(n_out / 128)][ceil(n_in / 128)], of one row: [ceil(n_in / 128)][n_out]
  bool w_rows;            // blocks of one row
  int64_t n_out;
  Epilogue ep;
  void* Y;
  bool y_bf16;
  void* workspace;
};

// Chooses the kernel of a call with M >= 1 rows by its sizes and types; false when a launch would exceed the dispatch limits.
struct Fp8Plan {
  bool quantize;  // X is quantised to the workspace first
  int rows, tokens;
  int stages = 2;  // of tiles of 128 x 128: steps in LDS
};
bool plan_fp8(const Fp8Call& c, Fp8Plan* plan);
size_t fp8_workspace_bytes(const Fp8Call& c, const Fp8Plan& plan);
hipError_t launch_fp8(const Fp8Call& c, const Fp8Plan& plan, hipStream_t stream);
// Its parts
bool fp8_few_grid_fits(const Fp8Call& c, int tokens);  // 16 or 32
bool fp8_few_quantizes(const Fp8Call& c, int tokens);  // X's tile fits its LDS
hipError_t launch_fp8_few(const Fp8Call& c, int tokens, hipStream_t stream);
bool fp8_tile_grid_fits(const Fp8Call& c, int rows, int tokens);
hipError_t launch_fp8_tile(const Fp8Call& c, int rows, int stages, hipStream_t stream);

// X [rows][cols] to e4m3 in blocks of 1 x 128 or 128 x 128 (`block`); the launch limits of that.
bool fp8_quantize_grids_fit(int64_t rows, int64_t cols, bool block, bool transposed);
hipError_t launch_fp8_quantize(const void* X, int64_t rows, int64_t cols, bool bf16, bool block, bool transposed, void* Q,
                               float* scales, hipStream_t stream);

#ifdef __HIPCC__
namespace {

constexpr float kE4m3Max = 448.0f, kLeastScale = 1.17549435e-38f;  // 2^-126

// A block's scale from its largest finite magnitude, and what entries are multiplied by: both divisions are rounded to
// nearest. The scale is a normal number, so its reciprocal is finite; no product passes 448 (1 + 2^-23), which rounds to 448.
__device__ __forceinline__ float block_scale(float amax) { return fmaxf(amax / kE4m3Max, kLeastScale); }

// Two entries, scaled, as e4m3 in the low or high half of `old` (hardware conversion, to nearest even)
template <bool HIGH>
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b, uint32_t old) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)old, HIGH);
}
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  return to_e4m3x2<true>(c, d, to_e4m3x2<false>(a, b, 0));
}
__device__ __forceinline__ uint32_t magnitude_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
constexpr uint32_t kInfBits = 0x7F800000u;

// Eight e4m3 entries as bfloat16 (exact: it has their exponents and more mantissa bits)
__device__ __forceinline__ bf16x8_t widen_e4m3(u32x2_t v) {
  u32x4_t w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.0f, false));
    w[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v[i], 1.0f, true));
  }
  return as_bf16x8(w);
}

// Eight consecutive entries of X as float32
template <bool BF16>
__device__ __forceinline__ void load8(const void* p, size_t at, float (&v)[8]) {
  if constexpr (BF16) {
    const u32x4_t w = *(const u32x4_t*)((const uint16_t*)p + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4_t w = ((const f32x4_t*)((const float*)p + at))[h];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * h + i] = w[i];
    }
  }
}

// The largest magnitude of N entries as its bits; a NaN or an infinity gives kInfBits or more.
template <int N>
__device__ __forceinline__ uint32_t largest_bits(const float (&v)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, magnitude_bits(v[i]));
  return m;
}
// Entries that are not finite become NaN (of which e4m3 has one) and no longer count: returns the largest finite magnitude.
template <int N>
__device__ __forceinline__ uint32_t drop_infinite(float (&v)[N]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t b = magnitude_bits(v[i]);
    if (b < kInfBits) m = max(m, b);
    else v[i] = __uint_as_float(0x7FC00000u);
  }
  return m;
}

}  // namespace
#endif
}  // namespace splr
