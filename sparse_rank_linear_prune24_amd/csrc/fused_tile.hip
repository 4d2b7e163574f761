// The layer product with a fused epilogue in workgroup tiles of 128 rows x 64 tokens, for one layer or for
// rows grouped by expert (LoSparse page, section 3.2, for the product): every size in float32 that the
// few-token kernel does not take, and in bfloat16 the sizes between it and the prefill kernel's 256 x 128
// tiles, which need thousands of tokens or outputs to occupy the chip.
//
// Four waves of 32 rows x 64 tokens. Per 64-column step X is staged in LDS by the workgroup (in float32
// as the three bfloat16 planes of fused_common.hpp, split once), S goes from memory to registers, both
// P steps ahead; the loads are raw buffer loads whose descriptors give zeros past the last row, column
// and step, so the loop has no branches and its last steps nothing special. The accumulators stay in
// registers; the rank-r term and the epilogue follow the loop.
//
// Why this tile: half of it (64 x 64) would read X from LDS twice as often per MFMA, twice of it leaves CUs
// without work at the sizes that come here. Measured, whole calls: bfloat16 4096 -> 4096 with 256 rows 31 us
// (the 256 x 128 tiles 50, the few-token kernel 68), 0.28 us a step and round of 256 tiles, bound by the
// latency of a step's LDS and barrier chain with one workgroup on a CU and by reading S and X through L2 with
// two; float32 4096 -> 4096 with 1000 rows 143 us (235 TFLOP/s of the dense product, above the float32 MFMA's
// 157), 1.0 us a step, of which 40 of the 48 MFMAs per wave are 0.18 us with one workgroup on a CU and
// 0.37 us with two, the splitting of S and X 0.3 us and the LDS reads next to nothing: the matrix cores and
// the vector ALUs hardly overlap here.
#include "common.hpp"
#include "epilogue.hpp"
#include "fused_common.hpp"
#include "groups.hpp"
#include "kernels.hpp"
#include "tile_common.hpp"

namespace splr {
namespace {

constexpr int kBuffer = 0x00020000;  // word 3 of a raw buffer descriptor: plain byte-addressed loads

template <bool F32>
struct TileType {
  using T = uint16_t;
  static constexpr int kParts = 1, kLead = 2, kSlots = 4, kBarrier = 2, kXAhead = 4, kSAhead = 8, kUnroll = 8;
};
// float32: a slot is three planes, and two workgroups share a CU's LDS
template <>
struct TileType<true> {
  using T = float;
  static constexpr int kParts = 3, kLead = 1, kSlots = 2, kBarrier = 1, kXAhead = 2, kSAhead = 2, kUnroll = 4;
};

template <bool F32, bool EXPERTS>
__global__ __launch_bounds__(256, 2) void fused_tile_kernel(
    const typename TileType<F32>::T* __restrict__ X, const typename TileType<F32>::T* __restrict__ values,
    const uint32_t* __restrict__ meta, const typename TileType<F32>::T* __restrict__ U, const float* __restrict__ T,
    int slices, Epilogue ep, void* Y, int y_bf16, int M, int K, int n_out, int r, int tiles_n, Groups groups) {
  using C = TileType<F32>;
  constexpr int NI = 2, NJ = 4, BM = 64, BN = 64 * NI;
  constexpr int kSize = F32 ? 4 : 2, kParts = C::kParts, PX = C::kXAhead, PS = C::kSAhead;
  constexpr int kUnroll = C::kUnroll;  // every ring index is constant; the steps past the last one multiply zeros
  constexpr int kPlane = BM * kXPitchU4;  // 16-byte units
  constexpr int kLanes = F32 ? 16 : 8;    // lanes that hold one token row of a step, 16 bytes each
  constexpr int kLoads = BM * kLanes / 256;
  // X of step kc + kLead is written during step kc: a barrier lies between (and between a slot's last
  // reads and its next writes) when both gaps span kBarrier steps
  static_assert(C::kLead >= C::kBarrier && C::kSlots - C::kLead >= C::kBarrier, "ring");
  static_assert(kUnroll % PX == 0 && kUnroll % PS == 0 && kUnroll % C::kSlots == 0 && kUnroll % 4 == 0, "constant ring indexes");
  constexpr int kTPitch = 68;  // floats of a row of 64 ranks
  __shared__ u32x4_t xs[C::kSlots][kParts * kPlane];
  __shared__ __align__(16) float ts[BM * kTPitch];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = lane & 15, quad = lane >> 4;
  const int TK = (K + 63) / 64, TKB = meta_blocks(TK), TR = (n_out + 15) / 16;
  // Each XCD (own L2) runs a contiguous range of the tiles, eight token tiles at a time row block by row
  // block, so that it reads S once for them and X once for its row blocks. Experts: all their tiles,
  // expert after expert.
  size_t e = 0, row0 = 0;
  const int t_rows = M;
  int tiles_m = (M + BM - 1) / BM;
  int tile;
  if constexpr (EXPERTS) {
    const int per_xcd = (group_tiles_total<BM>(groups) * tiles_n + 7) / 8;
    if ((int)(blockIdx.x >> 3) >= per_xcd) return;
    tile = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
    const GroupTile gt = find_group_tile<BM>(groups, tile / tiles_n);
    if (gt.expert < 0) return;
    tile -= gt.first * tiles_n;
    tiles_m = gt.tiles;
    M = gt.rows;
    e = gt.expert;
    row0 = gt.lo;
  } else {
    tile = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
    if (tile >= tiles_m * tiles_n) return;
  }
  constexpr int kGroupM = 8;
  const int group = tile / (kGroupM * tiles_n), in_group = tile - group * kGroupM * tiles_n;
  const int group_m = min(kGroupM, tiles_m - group * kGroupM);
  const int m_block = group * kGroupM + in_group % group_m, n_block = in_group / group_m;
  const int m0 = m_block * BM, n0 = n_block * BN + wave * 16 * NI;

  // X rows of the tile; a lane's 16 bytes of token row x_row + pass * (256 / kLanes)
  const int x_rows = min(BM, M - m0), x_end = x_rows * K * kSize;
  const __amdgpu_buffer_rsrc_t xrs =
      __builtin_amdgcn_make_buffer_rsrc((void*)(X + (row0 + m0) * K), (short)0, x_end, kBuffer);
  const int chunk = threadIdx.x % kLanes, x_row = threadIdx.x / kLanes;
  const int x_col = chunk * (16 / kSize);
  int x_off[kLoads];
#pragma unroll
  for (int t = 0; t < kLoads; ++t)
    x_off[t] = min(x_row + t * (256 / kLanes), x_rows - 1) * K * kSize + chunk * 16;
  // S and metadata of the wave's NI row fragments (fewer at the last tile row)
  constexpr int kTileBytes = 512 * kSize;
  const int tr0 = __builtin_amdgcn_readfirstlane(min(n0 / 16, TR - 1)), s_rows = min(NI, TR - tr0);
  const int s_stride = TK * kTileBytes, m_stride = TKB * 1024;
  const int s_end = s_rows * s_stride, m_end = s_rows * m_stride;
  const __amdgpu_buffer_rsrc_t srs = __builtin_amdgcn_make_buffer_rsrc(
      (void*)((const char*)values + (e * TR + tr0) * (size_t)s_stride), (short)0, s_end, kBuffer);
  const __amdgpu_buffer_rsrc_t mrs = __builtin_amdgcn_make_buffer_rsrc(
      (void*)((const char*)meta + (e * TR + tr0) * (size_t)m_stride), (short)0, m_end, kBuffer);

  u32x4_t xv[PX][kLoads], sv[PS][NI][F32 ? 2 : 1];
  uint32_t idx[kUnroll / 2][NI];  // a metadata word holds the indices of two steps
  auto load_x = [&](int kc, int t, u32x4_t& v) __attribute__((always_inline)) {
    const int away = kc * 64 + x_col >= K ? 1 << 30 : 0;  // past the row's end: past the descriptor's
    v = __builtin_amdgcn_raw_buffer_load_b128(xrs, x_off[t] + away, min(kc * 64 * kSize, x_end), 0);
  };
  auto store_x = [&](int slot, int t, u32x4_t v) __attribute__((always_inline)) {
    const int row = x_row + t * (256 / kLanes);
    if constexpr (F32) {
      const Parts4 q = split3(__builtin_bit_cast(f32x4_t, v));
#pragma unroll
      for (int k = 0; k < 3; ++k) ((u32x2_t*)xs[slot])[2 * (k * kPlane + row * kXPitchU4) + chunk] = q.p[k];
    } else {
      xs[slot][row * kXPitchU4 + chunk] = v;
    }
  };
  auto load_s = [&](int kc, int i, u32x4_t (&v)[F32 ? 2 : 1]) __attribute__((always_inline)) {
    const int so = kc < TK ? min(i * s_stride + kc * kTileBytes, s_end) : s_end;
#pragma unroll
    for (int h = 0; h < (F32 ? 2 : 1); ++h)
      v[h] = __builtin_amdgcn_raw_buffer_load_b128(srs, lane * (F32 ? 32 : 16) + 16 * h, so, 0);
  };
  auto load_m = [&](int kc, uint32_t (&w)[NI]) __attribute__((always_inline)) {  // kc even
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int so = kc < TK ? min(i * m_stride + (kc >> 3) * 1024 + 2 * (kc & 7), m_end) : m_end;
      w[i] = __builtin_amdgcn_raw_buffer_load_b32(mrs, lane * 16, so, 0);
    }
  };
  f32x4_t acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};
  // S as the product takes it: in float32 the parts of the present step and the next one's, split while the
  // present step's MFMAs run
  Parts8 a[2][NI];
  auto split_s = [&](const u32x4_t (&v)[F32 ? 2 : 1]) __attribute__((always_inline)) {
    if constexpr (F32)
      return split3(__builtin_bit_cast(f32x4_t, v[0]), __builtin_bit_cast(f32x4_t, v[F32 ? 1 : 0]));
    else
      return Parts8{{v[0], v[0], v[0]}};
  };

  auto step = [&](int kc, auto uu) __attribute__((always_inline)) {
    constexpr int u = decltype(uu)::value, slot = u % C::kSlots, xq = (u + C::kLead) % PX;
    bf16x16_t b[2][kParts];
    auto read_b = [&](int j) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < kParts; ++k) {
        const int at = k * kPlane + (16 * j + sub) * kXPitchU4 + quad;
        b[j & 1][k] = cat16(as_bf16x8(xs[slot][at]), as_bf16x8(xs[slot][at + 4]));
      }
    };
    read_b(0);
    __builtin_amdgcn_sched_barrier(0);
    // One group per token fragment: its MFMAs, the next fragment's LDS reads, and a part of the step's other
    // work, in float32 spread between the MFMAs (four vector instructions after each)
    static_for<NJ>([&](auto jj) __attribute__((always_inline)) {
      constexpr int j = decltype(jj)::value;
      if constexpr (j + 1 < NJ) read_b(j + 1);
      if constexpr (j < kLoads) {
        store_x((u + C::kLead) % C::kSlots, j, xv[xq][j]);
        load_x(kc + C::kLead + PX, j, xv[xq][j]);
      }
      if constexpr (F32 && j >= NJ - NI) {
        constexpr int i = j - (NJ - NI), ring = (u + 1) % PS;
        a[(u + 1) & 1][i] = split_s(sv[ring][i]);
        load_s(kc + 1 + PS, i, sv[ring][i]);
      }
      // S rows innermost, so that consecutive instructions write different accumulators; the products of
      // the small parts first
      constexpr int kTerms = F32 ? 6 : 1;
      constexpr int sp[6] = {F32 ? 2 : 0, 0, 1, 1, 0, 0}, xp[6] = {0, F32 ? 2 : 0, F32 ? 1 : 0, 0, F32 ? 1 : 0, 0};
#pragma unroll
      for (int t = 0; t < kTerms; ++t)
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const bf16x8_t s = as_bf16x8(F32 ? a[u & 1][i].p[sp[t]] : sv[u % PS][i][0]);
          acc[i][j] = smfmac16x16x64_half<u % 2>(s, b[j & 1][xp[t]], acc[i][j], idx[u / 2][i]);
        }
      if constexpr (F32) {
#pragma unroll
        for (int t = 0; t < kTerms * NI; ++t) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // an MFMA
          __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);  // vector instructions
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (!F32) {
#pragma unroll
      for (int i = 0; i < NI; ++i) load_s(kc + PS, i, sv[u % PS][i]);
    }
    if constexpr (u % 2 == 1) load_m(kc - 1 + kUnroll, idx[u / 2]);
    if constexpr (u % C::kBarrier == C::kBarrier - 1) lds_barrier();
  };

  // T's first 64 ranks (its K slices added) go to LDS before the loop, U's fragments of them to registers:
  // after it their latencies would be exposed
  const float* t_src = T + row0 * r;
  const typename C::T* u_src = U + e * n_out * r;
  TPairBuilder<BM, 256> tb;
  if (r > 0) {
    tb.init(t_src, slices, M, r, m0, 0, threadIdx.x, t_rows);
    tb.issue(0);
  }
  // rank block b of 16 (float32: ranks 16 b + 4 quad .. +3) or 32 (8 quad .. +7) ranks from j0 on
  constexpr int kRanks = F32 ? 16 : 32, kBlocks = 64 / kRanks;
  u32x4_t uv[NI][kBlocks];
  auto load_u = [&](int j0) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const int at = j0 + kRanks * b + (kRanks / 4) * quad;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const u32x4_t v = *(const u32x4_t*)(u_src + (size_t)min(n0 + 16 * i + sub, n_out - 1) * r + (at < r ? at : 0));
        uv[i][b] = at < r ? v : u32x4_t{0, 0, 0, 0};
      }
    }
  };
  if (r > 0) load_u(0);
  static_for<C::kLead>([&](auto v) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < kLoads; ++t) load_x(decltype(v)::value, t, xv[decltype(v)::value][t]);
  });
  static_for<PS>([&](auto v) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NI; ++i) load_s(decltype(v)::value, i, sv[decltype(v)::value][i]);
  });
  static_for<kUnroll / 2>([&](auto v) __attribute__((always_inline)) { load_m(2 * decltype(v)::value, idx[decltype(v)::value]); });
  __builtin_amdgcn_sched_barrier(0);
  if (r > 0) tb.finish_sums(ts, kTPitch);
  static_for<C::kLead>([&](auto v) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < kLoads; ++t) store_x(decltype(v)::value, t, xv[decltype(v)::value][t]);
  });
  static_for<PX>([&](auto v) __attribute__((always_inline)) {
    constexpr int kc = decltype(v)::value + C::kLead;
#pragma unroll
    for (int t = 0; t < kLoads; ++t) load_x(kc, t, xv[kc % PX][t]);
  });
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      a[0][i] = split_s(sv[0][i]);
      load_s(PS, i, sv[0][i]);
    }
  }
  lds_barrier();
  if (n0 < n_out) {
    for (int kc = 0; kc < TK; kc += kUnroll)
      static_for<kUnroll>([&](auto u) __attribute__((always_inline)) { step(kc + decltype(u)::value, u); });
  } else {  // a wave without rows (past the last one) only stages its share of X, with the same barriers
    for (int kc = 0; kc < TK; kc += kUnroll)
      static_for<kUnroll>([&](auto uu) __attribute__((always_inline)) {
        constexpr int u = decltype(uu)::value, xq = (u + C::kLead) % PX;
#pragma unroll
        for (int t = 0; t < kLoads; ++t) {
          store_x((u + C::kLead) % C::kSlots, t, xv[xq][t]);
          load_x(kc + u + C::kLead + PX, t, xv[xq][t]);
        }
        if constexpr (u % C::kBarrier == C::kBarrier - 1) lds_barrier();
      });
  }

  if constexpr (F32) {
    if (n0 < n_out)
      resum_nan(acc, X + row0 * K, values + (e * TR + n0 / 16) * (size_t)TK * 512,
                meta + (e * TR + n0 / 16) * (size_t)TKB * 256, K, M, n_out, n0, m0, sub, quad);
  }

  // acc += U T^T, 64 ranks at a time: in float32 on the float32 MFMA, in bfloat16 with T as three parts, so
  // that no rank is rounded
  for (int j0 = 0; j0 < r; j0 += 64) {
    if (j0 > 0) {
      load_u(j0);
      tb.init(t_src, slices, M, r, m0, j0, threadIdx.x, t_rows);
      tb.issue(0);
      lds_barrier();  // every wave has read the last block
      tb.finish_sums(ts, kTPitch);
      lds_barrier();
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      if (j0 + kRanks * b >= r) break;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float* p = ts + (16 * j + sub) * kTPitch + kRanks * b + (kRanks / 4) * quad;
        if constexpr (F32) {
          const f32x4_t t = *(const f32x4_t*)p;
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int i = 0; i < NI; ++i)
              acc[i][j] = mfma_f32(__builtin_bit_cast(f32x4_t, uv[i][b])[x], t[x], acc[i][j]);
        } else {
          const Parts8 t = split3(*(const f32x4_t*)p, *(const f32x4_t*)(p + 4));
#pragma unroll
          for (int k = 2; k >= 0; --k)
#pragma unroll
            for (int i = 0; i < NI; ++i) acc[i][j] = mfma16x16x32(as_bf16x8(uv[i][b]), as_bf16x8(t.p[k]), acc[i][j]);
        }
      }
    }
  }
  store_fragments<NI, NJ>(acc, ep, e * n_out, Y, y_bf16, M, n_out, n0, m0, row0, sub, quad);
}

int64_t tile_blocks(const FusedCall& c) { return c.offsets ? most_group_tiles(c.M, c.experts, 64) : ceil_div(c.M, 64); }

}  // namespace

bool fused_tile_grid_fits(const FusedCall& c) { return tile_blocks(c) * ceil_div(c.n_out, 128) < (int64_t(1) << 24); }

hipError_t launch_fused_tile(const FusedCall& c, hipStream_t stream) {
  const int tiles_n = (int)ceil_div(c.n_out, 128);
  const dim3 grid((unsigned)(8 * ceil_div(tiles_n * tile_blocks(c), 8)));
  const Groups groups{c.offsets, (int)c.experts, (int)c.M};
  const auto launch = [&](auto f32, auto kernel) {
    using T = typename TileType<decltype(f32)::value>::T;
    kernel<<<grid, dim3(256), 0, stream>>>((const T*)c.X, (const T*)c.values, c.meta, (const T*)c.U,
                                           (const float*)c.workspace, c.slices, c.ep, c.Y, c.y_bf16 ? 1 : 0, (int)c.M,
                                           (int)c.n_in, (int)c.n_out, (int)c.r, tiles_n, groups);
  };
  if (c.bf16)
    launch(std::false_type{}, c.offsets ? fused_tile_kernel<false, true> : fused_tile_kernel<false, false>);
  else
    launch(std::true_type{}, c.offsets ? fused_tile_kernel<true, true> : fused_tile_kernel<true, false>);
  return hipGetLastError();
}

}  // namespace splr
