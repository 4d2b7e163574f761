// The layer product with a fused epilogue, for one layer or for rows grouped by expert:
//   Z = X S^T + (X V^T) U^T + bias,  Y = act(Z) * gate + residual     (LoSparse page, section 3.2).
// Here: which kernels take a call, and the float32 kernels (one lane per output; a row's expert follows
// from the offsets). The bfloat16 kernels are those of the plain product with the epilogue in their
// last step (decode.hip, linear_bf16.hip).
#include <algorithm>

#include "common.hpp"
#include "epilogue.hpp"
#include "groups.hpp"
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
__global__ __launch_bounds__(256) void rows_lowrank_kernel(const float* __restrict__ X, const float* __restrict__ V,
                                                           const int32_t* __restrict__ offsets, int experts, int M,
                                                           int K, int r, float* __restrict__ T) {
  const int lane = threadIdx.x & 63;
  const int64_t outputs = (int64_t)M * r;
  for (int64_t o = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); o < outputs; o += (int64_t)gridDim.x * 4) {
    const int64_t m = o / r, j = o - m * r;
    const int e = expert_of_row(offsets, experts, (int)m);
    if (e < 0) continue;
    const float* x = X + (size_t)m * K;
    const float* v = V + ((size_t)e * r + j) * K;
    float t = 0.0f;
    for (int k = lane; k < K; k += 64) t = fmaf(x[k], v[k], t);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) t += __shfl_xor(t, off);
    if (lane == 0) T[o] = t;
  }
}

__global__ __launch_bounds__(256) void rows_fused_kernel(const float* __restrict__ X,
                                                         const float* __restrict__ values,
                                                         const uint32_t* __restrict__ meta,
                                                         const float* __restrict__ U, const float* __restrict__ T,
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
    const float* x = X + (size_t)m * K;
    float acc = 0.0f;
#pragma unroll 8
    for (int grp = 0; grp < K / 4; ++grp) {
      const int tk = grp / 16, gi = grp % 16, slot = n % 16 + 16 * (gi / 4);
      const uint32_t nib = (meta_unit(meta, TKB, tr, tk, slot) >> (4 * (gi % 4))) & 0xFu;
      const float* kept = values + ((size_t)tr * TK + tk) * 512 + slot * 8 + 2 * (gi % 4);
      acc = fmaf(x[4 * grp + (nib & 3u)], kept[0], acc);
      acc = fmaf(x[4 * grp + (nib >> 2)], kept[1], acc);
    }
    float lr = 0.0f;
    for (int j = 0; j < r; ++j) lr = fmaf(T[(size_t)m * r + j], U[((size_t)e * n_out + n) * r + j], lr);
    const size_t o = (size_t)m * n_out + n;
    const f32x4_t zero = {0, 0, 0, 0};
    const f32x4_t bias = ep.bias ? load4(ep.bias, (size_t)e * n_out + n, false, false, 1) : zero;
    const f32x4_t gate = ep.gate ? load4(ep.gate, o, y_bf16, false, 1) : zero;
    const f32x4_t residual = ep.residual ? load4(ep.residual, o, y_bf16, false, 1) : zero;
    const f32x4_t y = finish4(f32x4_t{acc + lr, 0, 0, 0}, bias, ep, gate, residual);
    store4<false>(Y, o, y_bf16, false, 1, y);
  }
}

constexpr int64_t kMaxBlocks = int64_t(1) << 20;

}  // namespace

namespace {

// Tokens that the decode kernel takes together, 0 where the prefill kernel is faster; for experts by the
// rows an expert has on average.
int decode_tokens(const FusedCall& c) {
  if (!c.offsets) return c.M <= kDecodeMaxTokens ? (int)c.M : 0;
  const int64_t mean = ceil_div(c.M, c.experts);
  if (mean <= 12) return 16;
  if (mean <= 24) return 32;
  return mean <= 64 ? 64 : 0;
}

dim3 rows_grid(const FusedCall& c) {
  return dim3((unsigned)std::min(ceil_div(c.n_out, 64) * ceil_div(c.M, 4), kMaxBlocks));
}

int slices_of(const FusedCall& c) {
  if (!c.bf16 || c.r == 0) return 1;
  return c.offsets ? experts_lowrank_slices(c) : lowrank_slices(c.M, c.n_in, c.r, true);
}

}  // namespace

size_t fused_workspace_bytes(const FusedCall& c) {
  return c.M == 0 || c.r == 0 ? 0 : (size_t)slices_of(c) * c.M * c.r * sizeof(float);
}

bool fused_grids_fit(const FusedCall& c) {
  if (!c.bf16) return true;  // both grids are capped
  if (c.r > 0 && !(c.offsets ? experts_lowrank_grid_fits(c) : lowrank_grids_fit(c.M, c.n_in, c.r, true))) return false;
  const int tokens = decode_tokens(c);
  if (!tokens) return fused_prefill_grid_fits(c);
  const int64_t block = tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64;
  return (c.offsets ? most_group_tiles(c.M, c.experts, block) : ceil_div(c.M, block)) <= 65535 &&
         grid_fits(dim3((unsigned)ceil_div(c.n_out, 16)), 256);
}

hipError_t launch_fused(FusedCall c, hipStream_t stream) {
  c.slices = slices_of(c);
  if (c.bf16) {
    if (c.r > 0) {
      const hipError_t e = c.offsets ? launch_experts_lowrank(c, stream)
                                     : launch_lowrank(c.X, c.V, c.M, c.n_in, c.r, true, c.workspace, stream);
      if (e != hipSuccess) return e;
    }
    const int tokens = decode_tokens(c);
    return tokens ? launch_fused_decode(c, tokens, stream) : launch_fused_prefill(c, stream);
  }
  float* T = (float*)c.workspace;
  if (c.r > 0) {
    const dim3 grid((unsigned)std::min(ceil_div(c.M * c.r, 4), kMaxBlocks));
    rows_lowrank_kernel<<<grid, dim3(256), 0, stream>>>((const float*)c.X, (const float*)c.V, c.offsets,
                                                        (int)c.experts, (int)c.M, (int)c.n_in, (int)c.r, T);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  rows_fused_kernel<<<rows_grid(c), dim3(256), 0, stream>>>(
      (const float*)c.X, (const float*)c.values, c.meta, (const float*)c.U, T, c.offsets, (int)c.experts, c.ep, c.Y,
      c.y_bf16 ? 1 : 0, (int)c.M, (int)c.n_in, (int)c.n_out, (int)c.r);
  return hipGetLastError();
}

}  // namespace splr
