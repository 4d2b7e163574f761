// The 8-bit product for few tokens: one workgroup 16 rows of W x 16 tokens, its waves the blocks of 128 columns in turn.
//
//   acc[n][m] += sx[m][kb] sw[n][kb] sum over k in block kb of W[n][k] X[m][k]
//
// Both operands become bfloat16 in registers (exact), so that the sums over a block are float32 sums on the bfloat16 matrix
// cores: reading W is what bounds this kernel, not its matrix instructions. X that is not held in 8 bits yet is quantised in
// registers, by the waves that use it: its blocks lie in one wave, and a launch of its own would cost more.
#include "fp8.hpp"

namespace splr {
namespace {

constexpr int kFewWaves = 8;
enum : int { kXe4m3 = 0, kXbf16 = 1, kXf32 = 2 };

template <int XT, bool EXPERTS>
__global__ __launch_bounds__(kFewWaves * kWave) void fp8_few_kernel(
    const void* __restrict__ X, const float* __restrict__ x_scales, const uint8_t* __restrict__ W,
    const float* __restrict__ w_scales, int w_rows, Epilogue ep, void* Y, int y_bf16, int M, int K, int n_out, Groups groups) {
  constexpr int kPitch = 20;  // floats of a token's 16 sums in LDS
  __shared__ __align__(16) float sums[kFewWaves][16 * kPitch];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = lane & 15, quad = lane >> 4;
  const int n0 = blockIdx.x * 16, KB = (K + kBlockK - 1) / kBlockK;
  size_t e = 0, row0 = 0;
  int rows = M, m0 = blockIdx.y * 16;
  if constexpr (EXPERTS) {
    const GroupTile gt = find_group_tile<16>(groups, blockIdx.y);
    if (gt.expert < 0) return;
    e = gt.expert;
    row0 = gt.lo;
    rows = gt.rows;
    m0 = (blockIdx.y - gt.first) * 16;
  }
  const int n = min(n0 + sub, n_out - 1);  // rows and tokens past the last are not stored
  const size_t m = row0 + min(m0 + sub, rows - 1);
  const uint8_t* w = W + (e * n_out + n) * K;
  const float* ws = w_scales + e * KB * (w_rows ? n_out : (n_out + 127) / 128);
  f32x4_t acc = {0, 0, 0, 0};
  for (int kb = wave; kb < KB; kb += kFewWaves) {
    // a lane's 32 columns of the block: 16 quad .. +15 and 64 + 16 quad .. +15
    const int c0 = kb * kBlockK + 16 * quad;
    const bool here[2] = {c0 < K, c0 + 64 < K};
    u32x4_t a[2], b[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) a[h] = here[h] ? *(const u32x4_t*)(w + c0 + 64 * h) : u32x4_t{0, 0, 0, 0};
    float sx;
    if constexpr (XT == kXe4m3) {
#pragma unroll
      for (int h = 0; h < 2; ++h) b[h] = here[h] ? *(const u32x4_t*)((const uint8_t*)X + m * K + c0 + 64 * h) : u32x4_t{0, 0, 0, 0};
      sx = x_scales[(size_t)kb * M + m];
    } else {
      float v[2][16];
      uint32_t most = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[h][i] = 0.0f;
        if (here[h]) load16<XT == kXbf16>(X, m * K + c0 + 64 * h, v[h]);
        most = max(most, largest_bits(v[h]));
      }
      if (__any(most >= kInfBits)) most = max(drop_infinite(v[0]), drop_infinite(v[1]));
      most = max(most, (uint32_t)__shfl_xor((int)most, 16));
      most = max(most, (uint32_t)__shfl_xor((int)most, 32));
      sx = block_scale(__uint_as_float(most));
      const float inv = 1.0f / sx;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          b[h][i] = to_e4m3x4(v[h][4 * i] * inv, v[h][4 * i + 1] * inv, v[h][4 * i + 2] * inv, v[h][4 * i + 3] * inv);
    }
    f32x4_t p = {0, 0, 0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        p = mfma16x16x32(widen_e4m3(u32x2_t{a[h][2 * i], a[h][2 * i + 1]}), widen_e4m3(u32x2_t{b[h][2 * i], b[h][2 * i + 1]}), p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = min(n0 + 4 * quad + i, n_out - 1);
      const float sw = w_rows ? ws[(size_t)kb * n_out + row] : ws[(size_t)(row / 128) * KB + kb];
      acc[i] = fmaf(p[i], sx * sw, acc[i]);
    }
  }
  // D fragment: token lane % 16, rows 4 (lane / 16) .. +3
  *(f32x4_t*)&sums[wave][sub * kPitch + 4 * quad] = acc;
  __syncthreads();
  if (wave > 0 || m0 + sub >= rows || n0 + 4 * quad >= n_out) return;
#pragma unroll
  for (int v = 1; v < kFewWaves; ++v) acc += *(const f32x4_t*)&sums[v][sub * kPitch + 4 * quad];
  const int row = n0 + 4 * quad, left = n_out - row;
  const bool vec = left >= 4 && n_out % 4 == 0;
  const size_t at = m * n_out + row;
  const f32x4_t none = {0, 0, 0, 0};
  const f32x4_t bias = ep.bias ? load4(ep.bias, e * n_out + row, ep.bias_bf16, vec, left) : none;
  const f32x4_t gate = ep.gate ? load4(ep.gate, at, y_bf16, vec, left) : none;
  const f32x4_t residual = ep.residual ? load4(ep.residual, at, y_bf16, vec, left) : none;
  store4<false>(Y, at, y_bf16, vec, left, finish4(acc, bias, ep, gate, residual));
}

dim3 few_grid(const Fp8Call& c) {
  return dim3((unsigned)ceil_div(c.n_out, 16),
              (unsigned)(c.offsets ? most_group_tiles(c.M, c.experts, 16) : ceil_div(c.M, 16)));
}

}  // namespace

bool fp8_few_grid_fits(const Fp8Call& c) { return grid_fits(few_grid(c), kFewWaves * kWave); }

hipError_t launch_fp8_few(const Fp8Call& c, hipStream_t stream) {
  const Groups groups{c.offsets, (int)c.experts, (int)c.M};
  const auto launch = [&](auto kernel) {
    kernel<<<few_grid(c), dim3(kFewWaves * kWave), 0, stream>>>(c.X, c.x_scales, c.W, c.w_scales, c.w_rows, c.ep, c.Y, c.y_bf16,
                                                                (int)c.M, (int)c.n_in, (int)c.n_out, groups);
  };
  if (c.x_type == 2) launch(c.offsets ? fp8_few_kernel<kXe4m3, true> : fp8_few_kernel<kXe4m3, false>);
  else if (c.x_type == 1) launch(c.offsets ? fp8_few_kernel<kXbf16, true> : fp8_few_kernel<kXbf16, false>);
  else launch(c.offsets ? fp8_few_kernel<kXf32, true> : fp8_few_kernel<kXf32, false>);
  return hipGetLastError();
}

}  // namespace splr
