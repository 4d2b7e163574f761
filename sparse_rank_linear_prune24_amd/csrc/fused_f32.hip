// The float32 layer product with a fused epilogue, for one layer or for rows grouped by expert:
//   Z = X S^T + (X V^T) U^T + bias,  Y = act(Z) * gate + residual     (LoSparse page, section 3.2).
//
// Here: the first stage and the kernel for few tokens. The sparse product takes every operand as three
// bfloat16 parts (fused_common.hpp); the thin products (T = X V^T and T U^T, a few percent of the work)
// use the float32 MFMA.
#include <algorithm>

#include "common.hpp"
#include "epilogue.hpp"
#include "fused_common.hpp"
#include "groups.hpp"
#include "kernels.hpp"
#include "tile_common.hpp"

namespace splr {
namespace {

// ------------------------------------------------------------------------------- first stage

// T = X V^T: a workgroup owns 16 tokens x 16 RF ranks over one K slice, its four waves take the slice's
// 64-column steps in turn (operands straight from memory: 64 contiguous bytes of a row per lane) and
// are added in wave order. Bound by latency and by reading X: 256 and more workgroups by slicing K.
template <int RF, bool EXPERTS>
__global__ __launch_bounds__(256) void f32_lowrank_kernel(const float* __restrict__ X, const float* __restrict__ V,
                                                          int M, int K, int r, int steps_per_slice,
                                                          float* __restrict__ part, Groups groups) {
  __shared__ f32x4_t red[3 * RF * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = lane & 15, quad = lane >> 4;
  int m_block = blockIdx.x;
  const size_t slice_rows = M;
  if constexpr (EXPERTS) {
    const GroupTile gt = find_group_tile<16>(groups, blockIdx.x);
    if (gt.expert < 0) return;
    m_block -= gt.first;
    M = gt.rows;
    X += (size_t)gt.lo * K;
    V += (size_t)gt.expert * r * K;
    part += (size_t)gt.lo * r;
  }
  const int m0 = m_block * 16, j0 = blockIdx.y * 16 * RF;
  const int TK = (K + 63) / 64;
  const int kb = blockIdx.z * steps_per_slice, ke = min(TK, kb + steps_per_slice);
  const float* x = X + (size_t)min(m0 + sub, M - 1) * K + 16 * quad;
  const float* v[RF];
#pragma unroll
  for (int a = 0; a < RF; ++a) v[a] = V + (size_t)min(j0 + 16 * a + sub, r - 1) * K + 16 * quad;
  f32x4_t acc[RF];
#pragma unroll
  for (int a = 0; a < RF; ++a) acc[a] = f32x4_t{0, 0, 0, 0};
  for (int kc = kb + wave; kc < ke; kc += 4) {
    const bool ok = kc * 64 + 16 * quad < K;  // a tail step holds 32 columns
    const int col = ok ? kc * 64 : 0;
    f32x4_t xv[4], vv[RF][4];
    const f32x4_t zero = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      xv[i] = *(const f32x4_t*)(x + col - (ok ? 0 : 16 * quad) + 4 * i);
#pragma unroll
      for (int a = 0; a < RF; ++a) vv[a][i] = *(const f32x4_t*)(v[a] + col - (ok ? 0 : 16 * quad) + 4 * i);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      xv[i] = ok ? xv[i] : zero;
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int a = 0; a < RF; ++a) acc[a] = mfma_f32(ok ? vv[a][i][e] : 0.0f, xv[i][e], acc[a]);
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int a = 0; a < RF; ++a) red[((wave - 1) * RF + a) * 64 + lane] = acc[a];
  }
  __syncthreads();
  if (wave != 0 || m0 + sub >= M) return;
  float* t = part + ((size_t)blockIdx.z * slice_rows + m0 + sub) * r;
#pragma unroll
  for (int a = 0; a < RF; ++a) {
#pragma unroll
    for (int w = 0; w < 3; ++w) acc[a] += red[(w * RF + a) * 64 + lane];
    const int j = j0 + 16 * a + 4 * quad;  // D rows: ranks; column: token
    if (j < r) *(f32x4_t*)(t + j) = acc[a];
  }
}

// U's and T's part of 16 ranks of the rank-r term: lane (sub, quad) holds ranks j0 + 4 quad .. +3 of row
// n0 + sub and of token m0 + 16 j + sub. All K slices of T (kMaxSlices at most) are requested together,
// clamped where there are fewer, and added in order.
constexpr int kMaxSlices = 8;
template <int NJ>
struct Ranks16 {
  f32x4_t u, t[NJ];
  __device__ __forceinline__ void load(const float* __restrict__ U, const float* __restrict__ T, size_t slice,
                                       int slices, int M, int n_out, int r, int j0, int n0, int m0, int sub, int quad) {
    u = *(const f32x4_t*)(U + (size_t)min(n0 + sub, n_out - 1) * r + j0 + 4 * quad);
    f32x4_t part[NJ][kMaxSlices];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int z = 0; z < kMaxSlices; ++z)
        part[j][z] = *(const f32x4_t*)(T + (size_t)min(m0 + 16 * j + sub, M - 1) * r + j0 + 4 * quad +
                                       (z < slices ? z : 0) * slice);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      t[j] = part[j][0];
#pragma unroll
      for (int z = 1; z < kMaxSlices; ++z) t[j] += z < slices ? part[j][z] : f32x4_t{0, 0, 0, 0};
    }
  }
  // acc[j] += U T^T on the float32 MFMA
  __device__ __forceinline__ void add(f32x4_t (&acc)[NJ]) const {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j] = mfma_f32(u[e], t[j][e], acc[j]);
  }
};

// A workgroup owns 16 rows x 16 NJ tokens; its four waves take the 64-column steps in turn, S and X
// straight from memory P steps ahead, and are added in wave order; wave 0 finishes, with the epilogue's
// operands and the first 16 ranks of U and T requested before the loop. Bound by reading S (2.1 KiB per 16 x
// 64 tile) and by latency: 6.3 us for 32 tokens 512 -> 512, where two launches and four dependent loads are all
// there is; 23 us a call for 16 tokens 4096 -> 4096 (38 MB of S and metadata).
template <int NJ, int P, bool EXPERTS>
__global__ __launch_bounds__(256) void f32_decode_kernel(const float* __restrict__ X, const float* __restrict__ values,
                                                         const uint32_t* __restrict__ meta,
                                                         const float* __restrict__ U, const float* __restrict__ T,
                                                         int slices, Epilogue ep, void* Y, int y_bf16, int M, int K,
                                                         int n_out, int r, Groups groups) {
  __shared__ f32x4_t red[3 * NJ * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = lane & 15, quad = lane >> 4;
  const int TK = (K + 63) / 64, TKB = meta_blocks(TK);
  int m_block = blockIdx.y;
  size_t e = 0, row0 = 0;
  const size_t slice = (size_t)M * r;
  if constexpr (EXPERTS) {
    const GroupTile gt = find_group_tile<16 * NJ>(groups, blockIdx.y);
    if (gt.expert < 0) return;
    m_block -= gt.first;
    M = gt.rows;
    e = gt.expert;
    row0 = gt.lo;
    X += row0 * K;
    T += row0 * r;
    U += e * n_out * r;
  }
  const int m0 = m_block * 16 * NJ, n0 = blockIdx.x * 16;
  const size_t tr = e * ((n_out + 15) / 16) + blockIdx.x;
  const float* s_src = values + tr * TK * 512 + lane * 8;
  const uint16_t* m_src = (const uint16_t*)meta + (tr * TKB * 64 + lane) * 8;
  const float* x_src[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) x_src[j] = X + (size_t)min(m0 + 16 * j + sub, M - 1) * K + 8 * quad;

  f32x4_t sv[P][2], xv[P][NJ][4];
  int idx[P];
  const int my_steps = (TK - wave + 3) / 4;  // this wave's steps are wave, wave + 4, ...
  // steps past the last one load the last one again and are not used
  auto load = [&](int s, int u) {
    const int kc = min(wave + 4 * s, TK - 1);
    sv[u][0] = __builtin_nontemporal_load((const f32x4_t*)(s_src + (size_t)kc * 512));
    sv[u][1] = __builtin_nontemporal_load((const f32x4_t*)(s_src + (size_t)kc * 512 + 4));
    idx[u] = m_src[(size_t)(kc >> 3) * 512 + (kc & 7)];
    const int up = kc * 64 + 32 < K ? 32 : 0;  // a tail step holds 32 columns: its upper half is zeroed below
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const float* x = x_src[j] + (size_t)kc * 64;
      xv[u][j][0] = *(const f32x4_t*)x;
      xv[u][j][1] = *(const f32x4_t*)(x + 4);
      xv[u][j][2] = *(const f32x4_t*)(x + up);
      xv[u][j][3] = *(const f32x4_t*)(x + up + 4);
    }
  };
  f32x4_t acc[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) acc[j] = f32x4_t{0, 0, 0, 0};
  const int n = n0 + 4 * quad, left = n_out - n;
  const bool vec = (n_out & 3) == 0 && left >= 4;
  f32x4_t bias = {0, 0, 0, 0}, gate[NJ], residual[NJ];
  Ranks16<NJ> ranks;
  static_for<P>([&](auto u) { load(decltype(u)::value, decltype(u)::value); });
  if (wave == 0) {
    if (r > 0) ranks.load(U, T, slice, slices, M, n_out, r, 0, n0, m0, sub, quad);
    if (ep.bias) bias = load4(ep.bias, e * n_out + n, false, vec, left);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const size_t at = (row0 + min(m0 + 16 * j + sub, M - 1)) * n_out + n;
      if (ep.gate) gate[j] = load4(ep.gate, at, y_bf16, vec, left);
      if (ep.residual) residual[j] = load4(ep.residual, at, y_bf16, vec, left);
    }
  }
  for (int s0 = 0; s0 < my_steps; s0 += P) {
    static_for<P>([&](auto uu) {
      constexpr int u = decltype(uu)::value;
      const int s = s0 + u, kc = wave + 4 * s;
      const Parts8 a = split3(sv[u][0], sv[u][1]);
      const int nib = idx[u];
      bf16x16_t b[NJ][3];
      const f32x4_t zero = {0, 0, 0, 0};
      const bool whole = kc * 64 + 32 < K;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const Parts8 lo = split3(xv[u][j][0], xv[u][j][1]);
        const Parts8 hi = split3(whole ? xv[u][j][2] : zero, whole ? xv[u][j][3] : zero);
#pragma unroll
        for (int k = 0; k < 3; ++k) b[j][k] = cat16(as_bf16x8(lo.p[k]), as_bf16x8(hi.p[k]));
      }
      if (s0 + P < my_steps) load(s + P, u);
      if (s < my_steps) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[j] = product6(a, b[j], nib, acc[j]);
      }
    });
  }
  if (wave > 0) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) red[((wave - 1) * NJ + j) * 64 + lane] = acc[j];
  }
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 0; w < 3; ++w)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[j] += red[(w * NJ + j) * 64 + lane];
  resum_nan<1, NJ>(reinterpret_cast<f32x4_t(&)[1][NJ]>(acc), X, values + tr * TK * 512, meta + tr * TKB * 256, K, M, n_out,
                   n0, m0, sub, quad);
  for (int j0 = 0; j0 < r; j0 += 16) {
    if (j0 > 0) ranks.load(U, T, slice, slices, M, n_out, r, j0, n0, m0, sub, quad);
    ranks.add(acc);
  }
  if (left <= 0) return;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int m = m0 + 16 * j + sub;
    const f32x4_t y = finish4(acc[j], bias, ep, gate[j], residual[j]);
    if (m < M) store4<false>(Y, (row0 + m) * n_out + n, y_bf16, vec, left, y);
  }
}

// ------------------------------------------------------------------------------- shapes

struct F32Stage1 {
  int rf, steps_per_slice, slices;
  dim3 grid;
};
F32Stage1 f32_stage1(const FusedCall& c) {
  F32Stage1 s;
  s.rf = c.r % 64 == 0 ? 4 : c.r % 32 == 0 ? 2 : 1;
  const int64_t blocks = c.offsets ? most_group_tiles(c.M, c.experts, 16) : ceil_div(c.M, 16);
  const int64_t TK = ceil_div(c.n_in, 64), others = c.r / (16 * s.rf);
  // K slices as far as they fill the chip, each at least a step for every wave; 8 at most, since every
  // workgroup of the second stage reads all of them
  const int64_t slices = std::min<int64_t>({kMaxSlices, ceil_div(TK, 4), std::max<int64_t>(1, 512 / (blocks * others))});
  s.steps_per_slice = (int)ceil_div(TK, slices);
  s.slices = (int)ceil_div(TK, s.steps_per_slice);
  s.grid = dim3((unsigned)blocks, (unsigned)others, (unsigned)s.slices);
  return s;
}

}  // namespace

int f32_lowrank_slices(const FusedCall& c) { return f32_stage1(c).slices; }
bool f32_lowrank_grid_fits(const FusedCall& c) { return grid_fits(f32_stage1(c).grid, 256); }

hipError_t launch_f32_lowrank(const FusedCall& c, hipStream_t stream) {
  const F32Stage1 s = f32_stage1(c);
  const Groups groups{c.offsets, (int)c.experts, (int)c.M};
  const auto launch = [&](auto kernel) {
    kernel<<<s.grid, dim3(256), 0, stream>>>((const float*)c.X, (const float*)c.V, (int)c.M, (int)c.n_in, (int)c.r,
                                             s.steps_per_slice, (float*)c.workspace, groups);
  };
  const bool experts = c.offsets != nullptr;
  if (s.rf == 4) launch(experts ? f32_lowrank_kernel<4, true> : f32_lowrank_kernel<4, false>);
  else if (s.rf == 2) launch(experts ? f32_lowrank_kernel<2, true> : f32_lowrank_kernel<2, false>);
  else launch(experts ? f32_lowrank_kernel<1, true> : f32_lowrank_kernel<1, false>);
  return hipGetLastError();
}

hipError_t launch_fused_decode_f32(const FusedCall& c, int tokens, hipStream_t stream) {
  const Groups groups{c.offsets, (int)c.experts, (int)c.M};
  const bool experts = c.offsets != nullptr;
  const dim3 grid((unsigned)ceil_div(c.n_out, 16),
                  (unsigned)(experts ? most_group_tiles(c.M, c.experts, tokens) : ceil_div(c.M, tokens)));
  const auto launch = [&](auto kernel) {
    kernel<<<grid, dim3(256), 0, stream>>>((const float*)c.X, (const float*)c.values, c.meta, (const float*)c.U,
                                           (const float*)c.workspace, c.slices, c.ep, c.Y, c.y_bf16 ? 1 : 0, (int)c.M,
                                           (int)c.n_in, (int)c.n_out, (int)c.r, groups);
  };
  if (tokens == 16) launch(experts ? f32_decode_kernel<1, 4, true> : f32_decode_kernel<1, 4, false>);
  else launch(experts ? f32_decode_kernel<2, 2, true> : f32_decode_kernel<2, 2, false>);
  return hipGetLastError();
}

}  // namespace splr
