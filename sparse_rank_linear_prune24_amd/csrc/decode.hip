// Y = X S^T + (X V^T) U^T for few tokens (M <= 64, bfloat16; LoSparse page, §3.2): the decode
// kernel. HBM-bound on S: a workgroup owns 16 rows (the fused forms
// also 32, NR = 2); its 4 waves take interleaved 64-column K steps,
// stream S straight into registers (non-temporal loads) and X through a private LDS slot each, and
// combine their partial accumulators through LDS in a fixed order; wave 0 adds the rank-r term and
// stores Y.
#include <algorithm>

#include "common.hpp"
#include "epilogue.hpp"
#include "groups.hpp"
#include "kernels.hpp"
#include "tile_common.hpp"

namespace splr {
namespace {

// ----------------------------------------------------------------------------------- decode

// U's rows tr0 + lane%16, ranks 16 (lane / 16) .. +15 of the first 64-rank block (zeros past n_out
// or r), as loaded; pair01 / pair23 give the (0,1) and (2,3) halves of every group of four ranks,
// the A operands of the two structured-sparse MFMAs that make one dense product
struct URow {
  u32x4_t d0, d1;
  __device__ __forceinline__ void load(const uint16_t* __restrict__ U, int n_out, int r, int tr0, int lane) {
    const int n = tr0 + (lane & 15), ju = 16 * (lane >> 4);
    const bool ok = n < n_out && ju < r;
    const uint16_t* p = U + (size_t)(ok ? n : 0) * r + (ok ? ju : 0);
    const u32x4_t zero = {0, 0, 0, 0};
    d0 = ok ? *(const u32x4_t*)p : zero;
    d1 = ok ? *(const u32x4_t*)(p + 8) : zero;
  }
  __device__ __forceinline__ bf16x8_t pair01() const { return as_bf16x8(u32x4_t{d0[0], d0[2], d1[0], d1[2]}); }
  __device__ __forceinline__ bf16x8_t pair23() const { return as_bf16x8(u32x4_t{d0[1], d0[3], d1[1], d1[3]}); }
};

// MODE: the plain product, with the fused epilogue, or that for rows grouped by expert (blockIdx.y is
// then a token block among all experts', and the operands are shifted to the block's expert and rows).
// The epilogue costs nothing measurable: one token 4096 -> 4096 with bias and residual takes 6.9 us after
// the first stage's 2.8, 16 gated tokens 4096 -> 14336 19 us a call (69 MB: 3.6 TB/s).
constexpr int kModePlain = 0, kModeFused = 1, kModeExperts = 2;

// NR: 16-row tiles a workgroup takes (fused modes): with two, each X fragment staged serves 32 rows.
// PADDED (fused modes): some wave's steps do not fill its ring, or the last step holds 32 columns. The launcher
// knows, so that full rings run without the tests of the last round (3 tokens 5504 -> 272: 12.5 -> 12.8 us with
// them; 333 tokens 1056 -> 1003, where whole steps fall away, 18.4 -> 17.9).
template <int MB, int P, int WAVES, int MODE = kModePlain, int NR = 1, bool PADDED = false>
__global__ __launch_bounds__(64 * WAVES) void linear_decode_kernel(
    const uint16_t* __restrict__ X_, const u32x4_t* __restrict__ values_, const uint32_t* __restrict__ meta_,
    const uint16_t* __restrict__ U_, const float* __restrict__ Tpart_, int slices, void* Y, int y_bf16, int M, int K,
    int n_out, int r, Epilogue ep, Groups groups) {
  int first_row = 0, m_block = blockIdx.y;
  size_t e = 0;
  if constexpr (MODE == kModeExperts) {
    const GroupTile gt = find_group_tile<16 * MB>(groups, blockIdx.y);
    if (gt.expert < 0) return;
    first_row = gt.lo;
    m_block = blockIdx.y - gt.first;
    M = gt.rows;
    e = gt.expert;
  }
  const size_t e_tiles = e * ((n_out + 15) / 16);  // tile rows before this expert's
  const uint16_t* __restrict__ X = X_ + (size_t)first_row * K;
  const u32x4_t* __restrict__ values = values_ + e_tiles * ((K + 63) / 64) * 64;
  const uint32_t* __restrict__ meta = meta_ + e_tiles * meta_blocks((K + 63) / 64) * 256;
  const uint16_t* __restrict__ U = U_ + e * n_out * r;
  const float* __restrict__ Tpart = Tpart_ + (size_t)first_row * r;
  constexpr int kXLoads = 2 * MB;  // 8 tokens x 128 bytes per load instruction, 16*MB tokens
  __shared__ u32x4_t xs[WAVES][16 * MB * kXPitchU4];
  __shared__ f32x4_t red[(WAVES - 1) * NR * MB * 64];
  __shared__ u32x4_t tpair[2 * kPreRankBlocks][16 * MB * kXPitchU4];  // T's bfloat16 pair (hi, lo)
  // the wave index is uniform across the wave; readfirstlane lets the compiler see that (scalar
  // loop control instead of exec-mask loops)
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = lane & 15, quad = lane >> 4;
  const int tr = blockIdx.x * NR, m0 = m_block * 16 * MB;
  const int TK = (K + 63) / 64;

  const u32x4_t* vsrc[NR];
  const uint16_t* msrc[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {  // a tile past the last one repeats it; never stored
    const int t = NR == 1 ? tr : min(tr + i, (n_out + 15) / 16 - 1);
    vsrc[i] = values + (size_t)t * TK * 64 + lane;
    msrc[i] = (const uint16_t*)meta + ((size_t)t * meta_blocks(TK) * 64 + lane) * 8;
  }
  const int xchunk = lane & 7;
  const uint16_t* xsrc[kXLoads];
  int xdst[kXLoads];
#pragma unroll
  for (int t = 0; t < kXLoads; ++t) {
    const int tloc = 8 * t + (lane >> 3);
    xsrc[t] = X + (size_t)min(m0 + tloc, M - 1) * K + 8 * xchunk;
    xdst[t] = tloc * kXPitchU4 + xchunk;
  }
  u32x4_t* st = xs[wave];

  f32x4_t acc[NR][MB];
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};

  // This wave's steps are kc = wave, wave + 4, ...; a ring of P steps of loads stays in flight:
  // slot u holds step s0 + u and is refilled with step s0 + u + P as soon as it has been consumed.
  // Branch-free: steps past the wave's last one load a clamped step and contribute through a
  // zeroed S operand. PADDED (fused modes) instead keeps an infinite X away from those zeros, whose product
  // would be NaN where the other fused kernels read zeros: in the last round, which alone holds such
  // steps, they are left out, and what a 32-column tail step re-reads is dropped.
  const int my_steps = (TK - wave + WAVES - 1) / WAVES;
  const int n_pad = max(1, (my_steps + P - 1) / P) * P;  // at least the final round (a wave may have no steps)
  u32x4_t sa[P][NR], xr[P][kXLoads];
  uint32_t sw[P][NR];
  auto load = [&](int s, u32x4_t (&va)[NR], uint32_t (&wa)[NR], u32x4_t (&xv)[kXLoads]) {
    const int kc = min(wave + s * WAVES, TK - 1);
    // S is read once per call: non-temporal, so it does not displace X, T and U, which every
    // workgroup re-reads (8.35 -> 7.85 us per 16-token call at 4096 x 4096)
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      va[i] = __builtin_nontemporal_load(vsrc[i] + (size_t)kc * 64);
      wa[i] = msrc[i][(size_t)(kc >> 3) * 512 + (kc & 7)];
    }
    int col = kc * 64;
    if (col + 8 * xchunk >= K) col -= 32;  // half tail step: re-read valid columns (S is zero there)
#pragma unroll
    for (int t = 0; t < kXLoads; ++t) xv[t] = *(const u32x4_t*)(xsrc[t] + col);
  };

  // T's pair: its loads go out first, the ring's next, and the pair is written to LDS while the
  // ring's loads are in flight (published by the barrier after the loop)
  const bool t_pre = r <= 64 * kPreRankBlocks;
  TPairBuilder<16 * MB, 64 * WAVES, MB == 1 ? 8 : 0> tb;  // 16 tokens: at most 8 K slices, all in one round
  if (t_pre && r > 0) {
    tb.init(Tpart, slices, M, r, m0, 0, threadIdx.x, MODE == kModeExperts ? groups.rows : 0);
    tb.issue(0);
  }
  // the epilogue's operands for the entries that wave 0 stores, loaded ahead like U's fragments: rows
  // n .. n+3 of token m0 + 16 j + lane % 16
  f32x4_t bias[NR], gate[NR][MB], residual[NR][MB];
  if constexpr (MODE != kModePlain) {
    if (wave == 0) {
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const int n = (tr + i) * 16 + 4 * quad, left = n_out - n;
        const bool vec = (n_out & 3) == 0 && left >= 4;
        bias[i] = ep.bias ? load4(ep.bias, e * n_out + n, ep.bias_bf16, vec, left) : f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < MB; ++j) {
          const size_t at = (size_t)(first_row + min(m0 + 16 * j + sub, M - 1)) * n_out + n;
          if (ep.gate) gate[i][j] = load4(ep.gate, at, y_bf16, vec, left);
          if (ep.residual) residual[i][j] = load4(ep.residual, at, y_bf16, vec, left);
        }
      }
    }
  }
  // U's fragments for wave 0's rank-r term, loaded now: after the loop their memory latency would
  // be exposed at the end of the call
  URow uf[NR];
  if (t_pre && r > 0 && wave == 0) {
#pragma unroll
    for (int i = 0; i < NR; ++i) uf[i].load(U, n_out, r, (tr + i) * 16, lane);
  }
  static_for<P>([&](auto uu) {  // issued in slot order (fenced), as the loop refills them
    constexpr int u = decltype(uu)::value;
    load(u, sa[u], sw[u], xr[u]);
    asm volatile("" ::: "memory");
  });
  if (t_pre && r > 0) tb.finish(tpair[0], tpair[1]);

  auto step = [&](int s, auto uu, auto refill) {
    constexpr int u = decltype(uu)::value;
    if constexpr (PADDED && !decltype(refill)::value) {
      if (s >= my_steps) return;  // wave-uniform
      if (wave + s * WAVES == TK - 1 && (K & 63) != 0 && xchunk >= 4) {
#pragma unroll
        for (int t = 0; t < kXLoads; ++t) xr[u][t] = u32x4_t{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int t = 0; t < kXLoads; ++t) st[xdst[t]] = xr[u][t];
    // wave-uniform; always all ones in the fused modes, where dropping it makes the compiler's schedule
    // slower (one token 4096 -> 4096 8.4 -> 9.0 us)
    const uint32_t keep = s < my_steps ? ~0u : 0u;
    bf16x8_t a[NR];
    int idx[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      a[i] = as_bf16x8(sa[u][i] & keep);
      idx[i] = (int)(sw[u][i] & keep);
    }
    if constexpr (decltype(refill)::value) load(s + P, sa[u], sw[u], xr[u]);
    // compiler-only fence: the refill stays in this step (not rotated into the next iteration,
    // which would shorten the prefetch distance of this slot)
    asm volatile("" ::: "memory");
#pragma unroll
    for (int j = 0; j < MB; ++j) {
      const int row = (16 * j + sub) * kXPitchU4;
      const bf16x16_t bx = cat16(as_bf16x8(st[row + quad]), as_bf16x8(st[row + 4 + quad]));
#pragma unroll
      for (int i = 0; i < NR; ++i) acc[i][j] = smfmac16x16x64(a[i], bx, acc[i][j], idx[i]);
    }
  };
  // every round but the last refills its slots; the last round loads nothing past the end
  for (int s0 = 0; s0 + P < n_pad; s0 += P)
    static_for<P>([&](auto uu) { step(s0 + decltype(uu)::value, uu, std::true_type{}); });
  static_for<P>([&](auto uu) { step(n_pad - P + decltype(uu)::value, uu, std::false_type{}); });

  // fixed-order combination of the waves' partial sums (into wave 0)
  if (wave > 0) {
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int j = 0; j < MB; ++j) red[(((wave - 1) * NR + i) * MB + j) * 64 + lane] = acc[i][j];
  }
  __syncthreads();
  if (wave == 0) {
#pragma unroll
    for (int w = 1; w < WAVES; ++w)
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] += red[(((w - 1) * NR + i) * MB + j) * 64 + lane];
  }
  // rank-r term, 64 ranks at a time: wave 0 adds U T^T, with T's pair from before the loop or, for
  // larger r, built block by block by all waves
  if (t_pre) {
    static_assert(kPreRankBlocks == 1, "one block of U fragments loaded ahead");
    if (wave == 0 && r > 0) {
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        const int row = (16 * j + sub) * kXPitchU4;
        const bf16x16_t th = cat16(as_bf16x8(tpair[0][row + quad]), as_bf16x8(tpair[0][row + 4 + quad]));
        const bf16x16_t tl = cat16(as_bf16x8(tpair[1][row + quad]), as_bf16x8(tpair[1][row + 4 + quad]));
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const bf16x8_t u01 = uf[i].pair01(), u23 = uf[i].pair23();
          acc[i][j] = smfmac16x16x64(u01, th, acc[i][j], 0x4444);
          acc[i][j] = smfmac16x16x64(u23, th, acc[i][j], 0xEEEE);
          acc[i][j] = smfmac16x16x64(u01, tl, acc[i][j], 0x4444);
          acc[i][j] = smfmac16x16x64(u23, tl, acc[i][j], 0xEEEE);
        }
      }
    }
  } else {
    for (int j0 = 0; j0 < r; j0 += 64) {
      build_t_pair<16 * MB, 64 * WAVES>(Tpart, slices, M, r, m0, j0, xs[0], xs[1], threadIdx.x,
                                        MODE == kModeExperts ? groups.rows : 0);
      lds_barrier();
      if (wave == 0) lowrank_block<NR, MB>(acc, U, xs[0], xs[1], n_out, r, j0, tr * 16, lane);
      lds_barrier();
    }
  }
  if (wave != 0) return;
  if constexpr (MODE == kModePlain) {
    store_tile<NR, MB>(acc, Y, y_bf16, M, n_out, tr * 16, m0, lane);
  } else {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int n = (tr + i) * 16 + 4 * quad, left = n_out - n;
      const bool vec = (n_out & 3) == 0 && left >= 4;
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        const int m = m0 + 16 * j + sub;
        if (m >= M) continue;
        const f32x4_t y = finish4(acc[i][j], bias[i], ep, gate[i][j], residual[i][j]);
        store4<false>(Y, (size_t)(first_row + m) * n_out + n, y_bf16, vec, left, y);
      }
    }
  }
}

dim3 decode_grid(int64_t M, int64_t n_out, int MB) {
  return dim3((unsigned)ceil_div(n_out, 16), (unsigned)ceil_div(M, 16 * MB));
}

template <int MB>
hipError_t launch_decode(const void* X, int64_t M, int64_t n_in, const void* values, const uint32_t* meta,
                         int64_t n_out, const void* U, int64_t r, const float* Tpart, int slices, void* Y,
                         int y_bf16, hipStream_t stream) {
  constexpr int P = MB == 1 ? 8 : 4, W = 4;
  const dim3 grid = decode_grid(M, n_out, MB);
  linear_decode_kernel<MB, P, W><<<grid, dim3(64 * W), 0, stream>>>(
      (const uint16_t*)X, (const u32x4_t*)values, meta, (const uint16_t*)U, Tpart, slices, Y, y_bf16, (int)M,
      (int)n_in, (int)n_out, (int)r, Epilogue{}, Groups{});
  return hipGetLastError();
}

// The load ring is as deep as the plain product's for one layer (8 steps of 16 tokens, 4 with two
// row tiles or 32 tokens) and 4 steps for experts, whose many workgroups then fit three to a CU: 32 experts 2048 -> 1024, two rows each, 26.5 ->
// 23.6 us (2 steps 22.3 there, but 62.6 -> 64.6 us for 4 experts 14336 -> 4096); one token 14336 -> 4096
// prefers the deeper ring, 20.1 against 20.7 us.
template <int MB, int NR>
hipError_t launch_fused_mb(const FusedCall& c, hipStream_t stream) {
  constexpr int P = MB == 1 && NR == 1 ? 8 : 4, W = 4;
  const bool experts = c.offsets != nullptr;
  const dim3 grid((unsigned)ceil_div(c.n_out, 16 * NR),
                  (unsigned)(experts ? most_group_tiles(c.M, c.experts, 16 * MB) : ceil_div(c.M, 16 * MB)));
  const auto launch = [&](auto kernel) {
    kernel<<<grid, dim3(64 * W), 0, stream>>>((const uint16_t*)c.X, (const u32x4_t*)c.values, c.meta,
                                              (const uint16_t*)c.U, (const float*)c.workspace, c.slices, c.Y,
                                              c.y_bf16 ? 1 : 0, (int)c.M, (int)c.n_in, (int)c.n_out, (int)c.r, c.ep,
                                              Groups{c.offsets, (int)c.experts, (int)c.M});
  };
  const auto rings_full = [&](int ring) { return c.n_in % (64 * W * ring) == 0; };
  if (experts && rings_full(4)) launch(linear_decode_kernel<MB, 4, W, kModeExperts, NR>);
  else if (experts) launch(linear_decode_kernel<MB, 4, W, kModeExperts, NR, true>);
  else if (rings_full(P)) launch(linear_decode_kernel<MB, P, W, kModeFused, NR>);
  else launch(linear_decode_kernel<MB, P, W, kModeFused, NR, true>);
  return hipGetLastError();
}

}  // namespace

bool decode_grids_fit(int64_t M, int64_t n_out) {
  return grid_fits(decode_grid(M, n_out, M <= 16 ? 1 : (M <= 32 ? 2 : 4)), 256);
}

hipError_t launch_linear_decode(const void* X, int64_t M, int64_t n_in, const void* values, const uint32_t* meta,
                                int64_t n_out, const void* U, int64_t r, const float* Tpart, int slices, void* Y,
                                bool y_bf16, hipStream_t stream) {
  const int yb = y_bf16 ? 1 : 0;
  if (M <= 16) return launch_decode<1>(X, M, n_in, values, meta, n_out, U, r, Tpart, slices, Y, yb, stream);
  if (M <= 32) return launch_decode<2>(X, M, n_in, values, meta, n_out, U, r, Tpart, slices, Y, yb, stream);
  return launch_decode<4>(X, M, n_in, values, meta, n_out, U, r, Tpart, slices, Y, yb, stream);
}

// Two row tiles a workgroup where that still leaves every CU one: each X fragment staged then serves 32
// rows. Measured, one / two (us): 16 tokens 4096 -> 14336 23.9 / 20.4, 4096 -> 8192 15.9 / 14.2, 8 experts 4096 ->
// 4096 of 8 rows 41.5 / 35.7; with half of the CUs left out 14336 -> 4096 24.2 / 30.2. 32 tokens: 4096 -> 8192
// 21.1 / 18.5, but short loops lose (333 rows 1056 -> 1003: 24.6 / 27.2).
bool few_token_pairs(const FusedCall& c, int64_t tokens) {
  const double active = (double)std::min(c.experts, c.M);
  const double blocks = c.offsets ? std::max(active, (double)c.M / tokens + active / 2) : (double)ceil_div(c.M, tokens);
  return c.bf16 && ceil_div(c.n_out, 32) * blocks >= 256 && (tokens == 16 || c.n_in >= 2048);
}

hipError_t launch_fused_decode(const FusedCall& c, int tokens, hipStream_t stream) {
  const bool pair = few_token_pairs(c, tokens);
  if (tokens == 16) return pair ? launch_fused_mb<1, 2>(c, stream) : launch_fused_mb<1, 1>(c, stream);
  return pair ? launch_fused_mb<2, 2>(c, stream) : launch_fused_mb<2, 1>(c, stream);
}

}  // namespace splr
