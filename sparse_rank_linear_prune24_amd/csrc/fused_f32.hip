// The float32 layer product with a fused epilogue, for one layer or for rows grouped by expert:
//   Z = X S^T + (X V^T) U^T + bias,  Y = act(Z) * gate + residual     (LoSparse page, section 3.2).
//
// The sparse product runs on the bfloat16 structured-sparse MFMA with float32 accuracy. A float32 number
// has 24 significant bits and a bfloat16 one 8, so x = x1 + x2 + x3 with x1 = RNE(x), x2 = RNE(x - x1),
// x3 = x - x1 - x2, all bfloat16 and the sum exact (|x| from about 1e-30 on; below, x3 may flush). Of the
// nine products of x1 + x2 + x3 and s1 + s2 + s3, each exact in the float32 accumulator, the six of
// order up to 2^-16 are summed; those left out, x2 s3, x3 s2 and x3 s3, are at most 2^-23 of x s (2^-25
// in the mean square), below the rounding of the float32 sum itself. Six structured-sparse MFMAs take
// about 117 cycles for 16 x 16 x 64 where the float32 MFMA needs 512 on an expanded S. An infinite X
// or S entry gives NaN (its low parts are infinity minus infinity).
// The thin products (T = X V^T and T U^T, a few percent of the work) use the float32 MFMA.
#include <algorithm>

#include "common.hpp"
#include "epilogue.hpp"
#include "groups.hpp"
#include "kernels.hpp"
#include "tile_common.hpp"

namespace splr {
namespace {

__device__ __forceinline__ f32x4_t mfma_f32(float a, float b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Eight float32 values as three bfloat16 parts (hardware conversion, to nearest even)
struct Parts8 {
  u32x4_t p[3];
};
__device__ __forceinline__ Parts8 split3(f32x4_t lo, f32x4_t hi) {
  Parts8 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f32x2_t x = i < 2 ? f32x2_t{lo[2 * i], lo[2 * i + 1]} : f32x2_t{hi[2 * i - 4], hi[2 * i - 3]};
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

// acc += S . X^T over one 64-column step, S and X in parts: the small products first
__device__ __forceinline__ f32x4_t product6(const Parts8& s, const bf16x16_t (&x)[3], int idx, f32x4_t acc) {
  acc = smfmac16x16x64(as_bf16x8(s.p[2]), x[0], acc, idx);
  acc = smfmac16x16x64(as_bf16x8(s.p[0]), x[2], acc, idx);
  acc = smfmac16x16x64(as_bf16x8(s.p[1]), x[1], acc, idx);
  acc = smfmac16x16x64(as_bf16x8(s.p[1]), x[0], acc, idx);
  acc = smfmac16x16x64(as_bf16x8(s.p[0]), x[1], acc, idx);
  return smfmac16x16x64(as_bf16x8(s.p[0]), x[0], acc, idx);
}

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

// acc[i][j] += U T^T over all ranks on the float32 MFMA, 16 ranks at a time: lane (sub, quad) holds ranks
// 4 quad .. +3 of row n0 + 16 i + sub and of token m0 + 16 j + sub. T's slices are added in order.
template <int NI, int NJ>
__device__ __forceinline__ void add_rank_term(f32x4_t (&acc)[NI][NJ], const float* __restrict__ U,
                                              const float* __restrict__ T, size_t slice, int slices, int M, int n_out,
                                              int r, int n0, int m0, int sub, int quad) {
  for (int j0 = 0; j0 < r; j0 += 16) {
    f32x4_t u[NI], t[NJ];
#pragma unroll
    for (int i = 0; i < NI; ++i) u[i] = *(const f32x4_t*)(U + (size_t)min(n0 + 16 * i + sub, n_out - 1) * r + j0 + 4 * quad);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const float* p = T + (size_t)min(m0 + 16 * j + sub, M - 1) * r + j0 + 4 * quad;
      t[j] = *(const f32x4_t*)p;
      for (int z = 1; z < slices; ++z) t[j] += *(const f32x4_t*)(p + z * slice);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[i][j] = mfma_f32(u[i][e], t[j][e], acc[i][j]);
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
    if (ep.bias) bias = load4(ep.bias, bias_row + n, false, vec, left);
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

// ------------------------------------------------------------------------------- few tokens

// A workgroup owns 16 rows x 16 NJ tokens; its four waves take the 64-column steps in turn, S and X
// straight from memory P steps ahead, and are added in wave order; wave 0 finishes. Bound by reading S
// (2.1 KiB per 16 x 64 tile) and by its latency.
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
  f32x4_t acc[1][NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) acc[0][j] = f32x4_t{0, 0, 0, 0};
  static_for<P>([&](auto u) { load(decltype(u)::value, decltype(u)::value); });
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
        for (int j = 0; j < NJ; ++j) acc[0][j] = product6(a, b[j], nib, acc[0][j]);
      }
    });
  }
  if (wave > 0) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) red[((wave - 1) * NJ + j) * 64 + lane] = acc[0][j];
  }
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int w = 0; w < 3; ++w)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[0][j] += red[(w * NJ + j) * 64 + lane];
  add_rank_term<1, NJ>(acc, U, T, slice, slices, M, n_out, r, n0, m0, sub, quad);
  store_fragments<1, NJ>(acc, ep, e * n_out, Y, y_bf16, M, n_out, n0, m0, row0, sub, quad);
}

// ------------------------------------------------------------------------------- many tokens

// Workgroup tile 64 NI rows x 64 tokens, four waves of 16 NI rows x 64 tokens. Per 64-column step X is
// split once by the workgroup and staged in LDS as three bfloat16 planes (two buffers, one barrier a
// step); every wave splits its own S rows in registers. Reading the planes costs each wave 24 KiB of
// LDS per step whatever its rows, so NI = 2 (128 rows) balances LDS and the matrix cores.
template <int NI, bool EXPERTS>
__global__ __launch_bounds__(256) void f32_tile_kernel(const float* __restrict__ X, const float* __restrict__ values,
                                                       const uint32_t* __restrict__ meta,
                                                       const float* __restrict__ U, const float* __restrict__ T,
                                                       int slices, Epilogue ep, void* Y, int y_bf16, int M, int K,
                                                       int n_out, int r, int tiles_n, Groups groups) {
  constexpr int NJ = 4, BM = 64, BN = 64 * NI;
  constexpr int kPlane = BM * kXPitchU4;  // 16-byte units
  __shared__ u32x4_t xs[2][3 * kPlane];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = lane & 15, quad = lane >> 4;
  const int TK = (K + 63) / 64, TKB = meta_blocks(TK), TR = (n_out + 15) / 16;
  int m_block = blockIdx.x / tiles_n;
  const int n_block = blockIdx.x - m_block * tiles_n;
  size_t e = 0, row0 = 0;
  const size_t slice = (size_t)M * r;
  if constexpr (EXPERTS) {
    const GroupTile gt = find_group_tile<BM>(groups, m_block);
    if (gt.expert < 0) return;
    m_block -= gt.first;
    M = gt.rows;
    e = gt.expert;
    row0 = gt.lo;
    X += row0 * K;
    T += row0 * r;
    U += e * n_out * r;
  }
  const int m0 = m_block * BM, n0 = n_block * BN + wave * 16 * NI;

  // X: thread t stages 16 columns (four lanes a row) of token row t / 4
  const int xr = threadIdx.x >> 2, xc = (threadIdx.x & 3) * 16;
  const float* x_src = X + (size_t)min(m0 + xr, M - 1) * K + xc;
  f32x4_t xv[4];
  auto load_x = [&](int kc) {
    const bool ok = kc < TK && kc * 64 + xc < K;
    const float* p = x_src + (ok ? kc * 64 : -xc);
    const f32x4_t zero = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4_t v = *(const f32x4_t*)(p + 4 * i);
      xv[i] = ok ? v : zero;
    }
  };
  auto store_x = [&](int buf) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const Parts8 q = split3(xv[2 * h], xv[2 * h + 1]);
#pragma unroll
      for (int k = 0; k < 3; ++k) xs[buf][k * kPlane + xr * kXPitchU4 + xc / 8 + h] = q.p[k];
    }
  };
  // S: the wave's row fragments (tile rows past the last repeat it; never stored)
  const float* s_src[NI];
  const uint16_t* m_src[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const size_t tr = e * TR + min(n0 / 16 + i, TR - 1);
    s_src[i] = values + tr * TK * 512 + lane * 8;
    m_src[i] = (const uint16_t*)meta + (tr * TKB * 64 + lane) * 8;
  }
  f32x4_t sv[NI][2];
  int idx[NI];
  auto load_s = [&](int kc) {
    kc = min(kc, TK - 1);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      sv[i][0] = *(const f32x4_t*)(s_src[i] + (size_t)kc * 512);
      sv[i][1] = *(const f32x4_t*)(s_src[i] + (size_t)kc * 512 + 4);
      idx[i] = m_src[i][(size_t)(kc >> 3) * 512 + (kc & 7)];
    }
  };
  f32x4_t acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};

  load_x(0);
  load_s(0);
  store_x(0);
  load_x(1);
  lds_barrier();
  for (int kc = 0; kc < TK; ++kc) {
    const int buf = kc & 1;
    Parts8 a[NI];
    int nib[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      a[i] = split3(sv[i][0], sv[i][1]);
      nib[i] = idx[i];
    }
    load_s(kc + 1);
    store_x(buf ^ 1);  // step kc + 1; that buffer's reads ended before the last barrier
    load_x(kc + 2);
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      bf16x16_t b[3];
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int at = k * kPlane + (16 * j + sub) * kXPitchU4 + quad;
        b[k] = cat16(as_bf16x8(xs[buf][at]), as_bf16x8(xs[buf][at + 4]));
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) acc[i][j] = product6(a[i], b, nib[i], acc[i][j]);
    }
    lds_barrier();
  }
  add_rank_term<NI, NJ>(acc, U, T, slice, slices, M, n_out, r, n0, m0, sub, quad);
  store_fragments<NI, NJ>(acc, ep, e * n_out, Y, y_bf16, M, n_out, n0, m0, row0, sub, quad);
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
  const int64_t slices = std::min<int64_t>({8, ceil_div(TK, 4), std::max<int64_t>(1, 512 / (blocks * others))});
  s.steps_per_slice = (int)ceil_div(TK, slices);
  s.slices = (int)ceil_div(TK, s.steps_per_slice);
  s.grid = dim3((unsigned)blocks, (unsigned)others, (unsigned)s.slices);
  return s;
}

}  // namespace

int fused_f32_slices(const FusedCall& c) { return c.r > 0 ? f32_stage1(c).slices : 1; }

bool fused_f32_grids_fit(const FusedCall& c, int tokens) {
  if (c.r > 0 && !grid_fits(f32_stage1(c).grid, 256)) return false;
  const int64_t tile = tokens ? (tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64) : 64;
  const int64_t m = c.offsets ? most_group_tiles(c.M, c.experts, tile) : ceil_div(c.M, tile);
  if (tokens) return m <= 65535 && grid_fits(dim3((unsigned)ceil_div(c.n_out, 16)), 256);
  return m * ceil_div(c.n_out, 128) < (int64_t(1) << 24);
}

hipError_t launch_fused_f32(const FusedCall& c, int tokens, hipStream_t stream) {
  const Groups groups{c.offsets, (int)c.experts, (int)c.M};
  const bool experts = c.offsets != nullptr;
  if (c.r > 0) {
    const F32Stage1 s = f32_stage1(c);
    const auto stage1 = [&](auto kernel) {
      kernel<<<s.grid, dim3(256), 0, stream>>>((const float*)c.X, (const float*)c.V, (int)c.M, (int)c.n_in, (int)c.r,
                                               s.steps_per_slice, (float*)c.workspace, groups);
    };
    if (s.rf == 4) stage1(experts ? f32_lowrank_kernel<4, true> : f32_lowrank_kernel<4, false>);
    else if (s.rf == 2) stage1(experts ? f32_lowrank_kernel<2, true> : f32_lowrank_kernel<2, false>);
    else stage1(experts ? f32_lowrank_kernel<1, true> : f32_lowrank_kernel<1, false>);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (tokens) {
    const int tile = tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64;
    const dim3 grid((unsigned)ceil_div(c.n_out, 16),
                    (unsigned)(experts ? most_group_tiles(c.M, c.experts, tile) : ceil_div(c.M, tile)));
    const auto decode = [&](auto kernel) {
      kernel<<<grid, dim3(256), 0, stream>>>((const float*)c.X, (const float*)c.values, c.meta, (const float*)c.U,
                                             (const float*)c.workspace, c.slices, c.ep, c.Y, c.y_bf16 ? 1 : 0,
                                             (int)c.M, (int)c.n_in, (int)c.n_out, (int)c.r, groups);
    };
    if (tile == 16) decode(experts ? f32_decode_kernel<1, 4, true> : f32_decode_kernel<1, 4, false>);
    else if (tile == 32) decode(experts ? f32_decode_kernel<2, 2, true> : f32_decode_kernel<2, 2, false>);
    else decode(experts ? f32_decode_kernel<4, 2, true> : f32_decode_kernel<4, 2, false>);
    return hipGetLastError();
  }
  const int tiles_n = (int)ceil_div(c.n_out, 128);
  const int64_t tiles_m = experts ? most_group_tiles(c.M, c.experts, 64) : ceil_div(c.M, 64);
  const auto kernel = experts ? f32_tile_kernel<2, true> : f32_tile_kernel<2, false>;
  kernel<<<dim3((unsigned)(tiles_n * tiles_m)), dim3(256), 0, stream>>>(
      (const float*)c.X, (const float*)c.values, c.meta, (const float*)c.U, (const float*)c.workspace, c.slices, c.ep,
      c.Y, c.y_bf16 ? 1 : 0, (int)c.M, (int)c.n_in, (int)c.n_out, (int)c.r, tiles_n, groups);
  return hipGetLastError();
}

}  // namespace splr
