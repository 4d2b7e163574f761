// The 8-bit product in large workgroup tiles, both operands through LDS.
//
//   acc[n][m] += sx[m][kb] sw[n][kb] p,   p = sum over the block's 128 columns of W[n][k] X[m][k]
//
// A step is one block of 128 columns: rows of 128 bytes of W and X go straight from memory to LDS (no registers between),
// two steps deep, and from there to the matrix instructions as fragments of 32 x 32. p starts from zero in every step, so
// that the scales can be applied to it in float32: 16 multiply-adds for every 32 x 32 x 128 products.
//
// Rows lie 128 bytes apart in LDS without padding (a direct load writes 64 consecutive pieces of 16 bytes); piece c of row r
// stands at place c ^ (r % 8) of its row, so that eight lanes that read one piece of eight rows meet all banks.
#include "fp8.hpp"
#include "tile_common.hpp"

namespace splr {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int kBuffer = 0x00020000;  // word 3 of a raw buffer descriptor: plain byte-addressed loads
constexpr int kAway = 1 << 30;       // past every descriptor's end: such a load gives zeros

// 16 or 4 bytes a lane from the buffer to LDS, lane after lane from `lds` on
template <int BYTES>
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t rs, uint8_t* lds, int offset, int step_offset) {
  if constexpr (BYTES == 16)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)lds, 16, offset, step_offset, 0, 0);
  else
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)lds, 4, offset, step_offset, 0, 0);
}

// All loads of this wave have arrived and its LDS reads are done, then workgroup barrier. The builtin wait is free; it
// tells the compiler that nothing is outstanding.
__device__ __forceinline__ void step_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0);
}

// 32 x 32 x 64 on e4m3 (the scaled form with no scales)
__device__ __forceinline__ f32x16_t mfma_e4m3(i32x8_t a, i32x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t mfma_bf16(bf16x8_t a, bf16x8_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// A fragment: a lane's 64 bytes of a step (row lane % 32; pieces 2 (lane / 32), + 1, + 4, + 5), as e4m3 or widened
template <bool WIDE>
struct Fragment;
template <>
struct Fragment<false> {
  i32x8_t v[2];
  __device__ __forceinline__ void set(const u32x4_t (&p)[4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[h][i] = (int)p[2 * h + i / 4][i % 4];
  }
};
template <>
struct Fragment<true> {
  bf16x8_t v[8];
  __device__ __forceinline__ void set(const u32x4_t (&p)[4]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = widen_e4m3(u32x2_t{p[i / 2][2 * (i & 1)], p[i / 2][2 * (i & 1) + 1]});
  }
};
__device__ __forceinline__ f32x16_t multiply(const Fragment<false>& a, const Fragment<false>& b) {
  f32x16_t p = {};
  p = mfma_e4m3(a.v[0], b.v[0], p);
  return mfma_e4m3(a.v[1], b.v[1], p);
}
__device__ __forceinline__ f32x16_t multiply(const Fragment<true>& a, const Fragment<true>& b) {
  f32x16_t p = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) p = mfma_bf16(a.v[i], b.v[i], p);
  return p;
}

// WR x WT waves, each NR x NT fragments of 32 rows of W x 32 tokens.
template <int WR, int WT, int NR, int NT>
struct Shape {
  static constexpr int kWaves = WR * WT, kThreads = kWaves * kWave, kRows = WR * NR * 32, kTokens = WT * NT * 32;
  static constexpr int kStage = (kRows + kTokens) * (kBlockK + 4);  // bytes of a step: both operands and their scales
  static constexpr int kPitch = NR * 32 + 4;                        // floats of a token's row in the epilogue
  static constexpr int kLds = 2 * kStage > kWaves * 32 * kPitch * 4 ? 2 * kStage : kWaves * 32 * kPitch * 4;
};

template <int WR, int WT, int NR, int NT, bool WIDE, bool W_ROWS, bool EXPERTS>
__global__ __launch_bounds__(WR * WT * kWave, 2) void fp8_tile_kernel(
    const uint8_t* __restrict__ X, const float* __restrict__ x_scales, const uint8_t* __restrict__ W,
    const float* __restrict__ w_scales, Epilogue ep, void* Y, int y_bf16, int M, int K, int n_out, int tiles_n, Groups groups) {
  using S = Shape<WR, WT, NR, NT>;
  constexpr int BN = S::kRows, BM = S::kTokens, kWaves = S::kWaves;
  __shared__ __align__(1024) uint8_t lds[S::kLds];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int KB = (K + kBlockK - 1) / kBlockK;
  // Each XCD (own L2) runs a contiguous range of the tiles, four token tiles at a time row block by row block, so that it
  // reads W once for them and X once for its row blocks. Experts: all their tiles, expert after expert.
  size_t e = 0, row0 = 0;
  const int all_rows = M;
  int tiles_m = (M + BM - 1) / BM, tile;
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
  constexpr int kGroupM = 4;
  const int group = tile / (kGroupM * tiles_n), in_group = tile - group * kGroupM * tiles_n;
  const int group_m = min(kGroupM, tiles_m - group * kGroupM);
  const int m0 = (group * kGroupM + in_group % group_m) * BM, n0 = in_group / group_m * BN;
  const int wave_n = wave / WT * NR * 32, wave_m = wave % WT * NT * 32;  // of the tile

  // What a wave loads: pieces of eight rows, a lane 16 bytes of one; rows past the last and columns past K come as zeros
  const int rows_n = min(BN, n_out - n0), rows_m = min(BM, M - m0);
  const __amdgpu_buffer_rsrc_t wrs =
      __builtin_amdgcn_make_buffer_rsrc((void*)(W + (e * n_out + n0) * K), (short)0, rows_n * K, kBuffer);
  const __amdgpu_buffer_rsrc_t xrs =
      __builtin_amdgcn_make_buffer_rsrc((void*)(X + (row0 + m0) * K), (short)0, rows_m * K, kBuffer);
  const int l_row = lane >> 3, l_col = ((lane & 7) ^ l_row) * 16;
  constexpr int kLoadsW = BN / 8 / kWaves, kLoadsX = BM / 8 / kWaves;
  static_assert(BN % (8 * kWaves) == 0 && BM % (8 * kWaves) == 0, "whole pieces");
  int w_off[kLoadsW], x_off[kLoadsX];
#pragma unroll
  for (int t = 0; t < kLoadsW; ++t) w_off[t] = (8 * (wave + kWaves * t) + l_row) * K + l_col;
#pragma unroll
  for (int t = 0; t < kLoadsX; ++t) x_off[t] = (8 * (wave + kWaves * t) + l_row) * K + l_col;
  constexpr int kX = BN * kBlockK, kScaleX = (BN + BM) * kBlockK, kScaleW = kScaleX + BM * 4;  // in a stage
  const float* const w_scale = w_scales + e * KB * (W_ROWS ? n_out : (n_out + 127) / 128);
  auto load = [&](int kb, int stage) __attribute__((always_inline)) {
    uint8_t* const to = lds + stage * S::kStage;
    if (kb == KB - 1 && K % kBlockK) {  // nothing is loaded after this step
      const int away = kb * kBlockK + l_col >= K ? kAway : 0;
#pragma unroll
      for (int t = 0; t < kLoadsW; ++t) w_off[t] += away;
#pragma unroll
      for (int t = 0; t < kLoadsX; ++t) x_off[t] += away;
    }
#pragma unroll
    for (int t = 0; t < kLoadsW; ++t) load_to_lds<16>(wrs, to + (wave + kWaves * t) * 1024, w_off[t], kb * kBlockK);
#pragma unroll
    for (int t = 0; t < kLoadsX; ++t) load_to_lds<16>(xrs, to + kX + (wave + kWaves * t) * 1024, x_off[t], kb * kBlockK);
    if (wave < BM / 64) {
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(x_scales + (size_t)kb * all_rows + row0 + m0), (short)0, rows_m * 4, kBuffer);
      load_to_lds<4>(rs, to + kScaleX + wave * 256, (wave * 64 + lane) * 4, 0);
    } else if (W_ROWS && wave - BM / 64 < BN / 64) {
      const __amdgpu_buffer_rsrc_t rs =
          __builtin_amdgcn_make_buffer_rsrc((void*)(w_scale + (size_t)kb * n_out + n0), (short)0, rows_n * 4, kBuffer);
      load_to_lds<4>(rs, to + kScaleW + (wave - BM / 64) * 256, ((wave - BM / 64) * 64 + lane) * 4, 0);
    }
  };
  static_assert(!W_ROWS || BM / 64 + BN / 64 <= kWaves, "a wave for each 64 scales");

  const int sub = lane & 31, half = lane >> 5;
  // a lane's four pieces of its row: 2 half, 2 half + 1, and those + 4
  int at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) at[i] = sub * kBlockK + (((2 * half + (i & 1) + 4 * (i >> 1)) ^ (sub & 7)) * 16);
  auto read = [&](const uint8_t* rows, u32x4_t (&p)[4]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = *(const u32x4_t*)(rows + at[i]);
  };

  f32x16_t acc[NR][NT];
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x16_t{};
  const float* sw_block = w_scale + (size_t)(min(n0 + wave_n, n_out - 1) / 128) * KB;
  load(0, 0);
  for (int kb = 0; kb < KB; ++kb) {
    const int stage = kb & 1;
    const float sw = W_ROWS ? 1.0f : sw_block[kb];
    step_barrier();
    if (kb + 1 < KB) load(kb + 1, stage ^ 1);
    const uint8_t* const w = lds + stage * S::kStage + wave_n * kBlockK;
    const uint8_t* const x = lds + stage * S::kStage + kX + wave_m * kBlockK;
    const float* const sx = (const float*)(lds + stage * S::kStage + kScaleX) + wave_m + sub;
    const float* const sr = (const float*)(lds + stage * S::kStage + kScaleW) + wave_n + 4 * half;
    float s[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) s[j] = sx[32 * j] * sw;
    Fragment<WIDE> a[NR], b[2];
    u32x4_t raw[4];
    read(w, raw);
    a[0].set(raw);
    read(x, raw);
    b[0].set(raw);
#pragma unroll
    for (int i = 1; i < NR; ++i) {
      read(w + i * 32 * kBlockK, raw);
      a[i].set(raw);
    }
    // One group for each fragment of the result: its matrix instructions, and while they run the multiply-adds of the one
    // before and the reads of the next column of fragments
    f32x16_t p[2];
    auto scale = [&](int i, int j, const f32x16_t& q) __attribute__((always_inline)) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if constexpr (W_ROWS) {
          const f32x4_t r = *(const f32x4_t*)(sr + 32 * i + 8 * g);
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[i][j][4 * g + k] = fmaf(q[4 * g + k], s[j] * r[k], acc[i][j][4 * g + k]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[i][j][4 * g + k] = fmaf(q[4 * g + k], s[j], acc[i][j][4 * g + k]);
        }
      }
    };
    static_for<NR * NT>([&](auto tt) __attribute__((always_inline)) {
      constexpr int t = decltype(tt)::value, i = t % NR, j = t / NR;
      if constexpr (i == 0 && j + 1 < NT) read(x + (j + 1) * 32 * kBlockK, raw);
      p[t & 1] = multiply(a[i], b[j & 1]);
      if constexpr (t > 0) scale((t - 1) % NR, (t - 1) / NR, p[(t - 1) & 1]);
      if constexpr (i == NR - 1 && j + 1 < NT) b[(j + 1) & 1].set(raw);
      constexpr int kInstructions = WIDE ? 8 : 2, kEach = WIDE ? 4 : 8;
#pragma unroll
      for (int k = 0; k < kInstructions; ++k) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);      // a matrix instruction
        __builtin_amdgcn_sched_group_barrier(0x002, kEach, 0);  // vector instructions
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    scale(NR - 1, NT - 1, p[(NR * NT - 1) & 1]);
  }
  // The result through LDS, 32 tokens at a time in a part of each wave's own, so that loads and stores of the epilogue take
  // whole token rows of the wave's 32 NR outputs. D fragment: token lane % 32, rows 8 g + 4 (lane / 32) .. + 3.
  step_barrier();
  constexpr int kLanes = NR * 8, kRound = kWave / kLanes;  // lanes a token row, tokens at a time
  float* const mine = (float*)lds + wave * 32 * S::kPitch;
  const int c = lane % kLanes * 4, n = n0 + wave_n + c, left = n_out - n;
  const bool vec = left >= 4 && n_out % 4 == 0;
  const f32x4_t none = {0, 0, 0, 0};
  const f32x4_t bias = ep.bias && left > 0 ? load4(ep.bias, e * n_out + n, ep.bias_bf16, vec, left) : none;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *(f32x4_t*)(mine + sub * S::kPitch + 32 * i + 8 * g + 4 * half) =
            f32x4_t{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int r = 0; r < 32; r += kRound) {
      const int token = r + lane / kLanes, m = m0 + wave_m + 32 * j + token;
      const f32x4_t sum = *(const f32x4_t*)(mine + token * S::kPitch + c);
      if (m < M && left > 0) {
        const size_t where = (row0 + m) * n_out + n;
        const f32x4_t gate = ep.gate ? load4(ep.gate, where, y_bf16, vec, left) : none;
        const f32x4_t residual = ep.residual ? load4(ep.residual, where, y_bf16, vec, left) : none;
        store4<false>(Y, where, y_bf16, vec, left, finish4(sum, bias, ep, gate, residual));
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

int64_t tile_blocks(const Fp8Call& c, int tokens) {
  return c.offsets ? most_group_tiles(c.M, c.experts, tokens) : ceil_div(c.M, tokens);
}

template <int WR, int WT, int NR, int NT, bool WIDE>
hipError_t launch_shape(const Fp8Call& c, hipStream_t stream) {
  using S = Shape<WR, WT, NR, NT>;
  const int tiles_n = (int)ceil_div(c.n_out, S::kRows);
  const dim3 grid((unsigned)(8 * ceil_div(tiles_n * tile_blocks(c, S::kTokens), 8)));
  const Groups groups{c.offsets, (int)c.experts, (int)c.M};
  const auto launch = [&](auto kernel) {
    kernel<<<grid, dim3(S::kThreads), 0, stream>>>((const uint8_t*)c.X, c.x_scales, c.W, c.w_scales, c.ep, c.Y, c.y_bf16 ? 1 : 0,
                                                   (int)c.M, (int)c.n_in, (int)c.n_out, tiles_n, groups);
  };
  if (c.w_rows) launch(c.offsets ? fp8_tile_kernel<WR, WT, NR, NT, WIDE, true, true> : fp8_tile_kernel<WR, WT, NR, NT, WIDE, true, false>);
  else launch(c.offsets ? fp8_tile_kernel<WR, WT, NR, NT, WIDE, false, true> : fp8_tile_kernel<WR, WT, NR, NT, WIDE, false, false>);
  return hipGetLastError();
}

}  // namespace

bool fp8_tile_grid_fits(const Fp8Call& c, int rows, int tokens) {
  return tile_blocks(c, tokens) * ceil_div(c.n_out, rows) < (int64_t(1) << 23);
}

hipError_t launch_fp8_tile(const Fp8Call& c, int rows, hipStream_t stream) {
  if (rows == 256) return c.y_bf16 ? launch_shape<4, 2, 2, 4, false>(c, stream) : launch_shape<4, 2, 2, 2, true>(c, stream);
  return c.y_bf16 ? launch_shape<2, 2, 2, 2, false>(c, stream) : launch_shape<2, 2, 2, 2, true>(c, stream);
}

}  // namespace splr
