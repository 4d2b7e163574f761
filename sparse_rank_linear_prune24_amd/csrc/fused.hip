// The layer product with a fused epilogue, for one layer or for rows grouped by expert:
//   Z = X S^T + (X V^T) U^T + bias,  Y = act(Z) * gate + residual     (LoSparse page, section 3.2).
// One lane per output, for every type and size; a row's expert follows from the offsets.
#include <algorithm>

#include "common.hpp"
#include "epilogue.hpp"
#include "kernels.hpp"

namespace splr {
namespace {

// The expert of row m: the last e with offsets[e] <= m, or -1 where no group holds m. Whatever the
// offsets hold, the result is -1 or a valid expert.
__device__ __forceinline__ int expert_of_row(const int32_t* __restrict__ offsets, int experts, int m) {
  if (!offsets) return 0;
  int lo = 0, hi = experts;  // offsets[lo] <= m < offsets[hi], once both ends are checked
  if (m < offsets[0] || m >= offsets[experts]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (offsets[mid] <= m) lo = mid;
    else hi = mid;
  }
  return lo;
}

// T[m][j] = X[m] . V_e[j], one wave per output
template <bool BF16>
__global__ __launch_bounds__(256) void rows_lowrank_kernel(const void* __restrict__ X, const void* __restrict__ V,
                                                           const int32_t* __restrict__ offsets, int experts, int M,
                                                           int K, int r, float* __restrict__ T) {
  const int lane = threadIdx.x & 63;
  const int64_t outputs = (int64_t)M * r;
  for (int64_t o = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); o < outputs; o += (int64_t)gridDim.x * 4) {
    const int64_t m = o / r, j = o - m * r;
    const int e = expert_of_row(offsets, experts, (int)m);
    if (e < 0) continue;
    float t = 0.0f;
    for (int k = lane; k < K; k += 64)
      t = fmaf(load_as_float(X, (size_t)m * K + k, BF16), load_as_float(V, ((size_t)e * r + j) * K + k, BF16), t);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) t += __shfl_xor(t, off);
    if (lane == 0) T[o] = t;
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void rows_fused_kernel(const void* __restrict__ X, const void* __restrict__ values,
                                                         const uint32_t* __restrict__ meta,
                                                         const void* __restrict__ U, const float* __restrict__ T,
                                                         const int32_t* __restrict__ offsets, int experts,
                                                         Epilogue ep, void* Y, int y_bf16, int M, int K, int n_out,
                                                         int r) {
  const int64_t nb = (n_out + 63) / 64, tiles = nb * ((M + 3) / 4);
  const int TK = (K + 63) / 64, TKB = meta_blocks(TK), TR = (n_out + 15) / 16;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int n = (int)(t % nb) * 64 + (threadIdx.x & 63);
    const int m = (int)(t / nb) * 4 + (threadIdx.x >> 6);
    if (n >= n_out || m >= M) continue;
    const int e = expert_of_row(offsets, experts, m);
    if (e < 0) continue;
    const int64_t tr = (int64_t)e * TR + n / 16;
    float acc = 0.0f;
#pragma unroll 8
    for (int grp = 0; grp < K / 4; ++grp) {
      const int tk = grp / 16, gi = grp % 16, slot = n % 16 + 16 * (gi / 4);
      const uint32_t nib = (meta_unit(meta, TKB, tr, tk, slot) >> (4 * (gi % 4))) & 0xFu;
      const size_t kept = ((size_t)tr * TK + tk) * 512 + slot * 8 + 2 * (gi % 4);
      const size_t x = (size_t)m * K + 4 * grp;
      acc = fmaf(load_as_float(X, x + (nib & 3u), BF16), load_as_float(values, kept, BF16), acc);
      acc = fmaf(load_as_float(X, x + (nib >> 2), BF16), load_as_float(values, kept + 1, BF16), acc);
    }
    float lr = 0.0f;
    for (int j = 0; j < r; ++j)
      lr = fmaf(T[(size_t)m * r + j], load_as_float(U, ((size_t)e * n_out + n) * r + j, BF16), lr);
    const size_t o = (size_t)m * n_out + n;
    float y = acc + lr;
    if (ep.bias) y += load_as_float(ep.bias, (size_t)e * n_out + n, BF16);
    y = activate(y, ep.act);
    if (ep.gate) y *= load_as_float(ep.gate, o, y_bf16);
    if (ep.residual) y += load_as_float(ep.residual, o, y_bf16);
    if (y_bf16) ((uint16_t*)Y)[o] = (uint16_t)float_to_bf16_bits(y);
    else ((float*)Y)[o] = y;
  }
}

constexpr int64_t kMaxBlocks = int64_t(1) << 20;

}  // namespace

size_t fused_workspace_bytes(int64_t M, int64_t r) { return (size_t)M * r * sizeof(float); }

hipError_t launch_fused(const void* X, int64_t M, int64_t n_in, const int32_t* offsets, int64_t experts,
                        const void* values, const uint32_t* meta, int64_t n_out, const void* U, const void* V,
                        int64_t r, bool bf16, const Epilogue& ep, void* Y, bool y_bf16, void* workspace,
                        hipStream_t stream) {
  float* T = (float*)workspace;
  if (r > 0) {
    const dim3 grid((unsigned)std::min(ceil_div(M * r, 4), kMaxBlocks));
    const auto stage1 = bf16 ? rows_lowrank_kernel<true> : rows_lowrank_kernel<false>;
    stage1<<<grid, dim3(256), 0, stream>>>(X, V, offsets, (int)experts, (int)M, (int)n_in, (int)r, T);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)std::min(ceil_div(n_out, 64) * ceil_div(M, 4), kMaxBlocks));
  const auto stage2 = bf16 ? rows_fused_kernel<true> : rows_fused_kernel<false>;
  stage2<<<grid, dim3(256), 0, stream>>>(X, values, meta, U, T, offsets, (int)experts, ep, Y, y_bf16 ? 1 : 0, (int)M,
                                         (int)n_in, (int)n_out, (int)r);
  return hipGetLastError();
}

}  // namespace splr
