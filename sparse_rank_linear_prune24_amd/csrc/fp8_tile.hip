// The 8-bit product in workgroup tiles of 128 x 128 and 256 x 256, both operands through LDS.
//
//   acc[n][m] += sx[m][kb] sw[n][kb] p,   p = sum over the block's 128 columns of W[n][k] X[m][k]
//
// A step is one block of 128 columns: rows of 128 bytes of W and X go straight from memory to LDS (no registers between), two
// or four steps deep, and from there to the matrix instructions as fragments of 32 x 32. p starts from zero in every step, so
// that the scales can be applied to it in float32: 16 multiply-adds a lane for every 32 x 32 x 128 products.
//
// With a bfloat16 Y the products run on the e4m3 matrix instructions. Of each eight consecutive products these keep what lies
// within 2^-13 of the largest (measured: one 2^-14 of it is lost), a loss of 2^-15 of the result's norm, which rounding Y (2^-9
// of it) hides. A float32 Y would show it, so for that both operands are widened to bfloat16, exactly, on their way from LDS, and
// the sums of a block are float32 sums, at half the rate.
//
// What bounds it, 8192 x 4096 -> 14336, bfloat16 Y, 480 us (2.0 PFLOP/s; the matrix instructions alone with their multiply-adds
// run at 4.4): the power limit holds the clock at 1.7 GHz, of whose cycles the matrix cores take 59 %; the same loop without
// its loads from memory takes 403 us, and about 70 us are the fills and epilogues of seven rounds of tiles, which n_in does not
// change (n_in 2048: 274 us, 8192: 865). 16 x 16 x 128 instructions instead of 32 x 32 x 64: 605 us at the time
// when these took 550; four multiply-adds an instruction leave no room between dependent ones. One word of each line fetched two
// steps ahead (for L2): 8 % slower, the requests are what is short. A float32 Y: 905 us (1.06 PFLOP/s), bound by the conversions
// (32 for every 8 matrix instructions, 1.5 times the time of other vector instructions) beside them.
//
// Rows lie 128 bytes apart in LDS without padding (a direct load writes 64 consecutive pieces of 16 bytes); piece c of row r
// stands at place c ^ (r / 2 % 8) of its row, so that the 16 lanes that read 16 bytes each at a time (lanes 0 .. 3, 12 .. 15,
// 20 .. 27 and 4 .. 11, 16 .. 19, 28 .. 31 of each half) meet every bank once.
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

// All loads of this wave but the last `LATER` have arrived and its LDS reads are done, then workgroup barrier. The builtin wait
// is free; it tells the compiler what is outstanding.
template <int LATER>
__device__ __forceinline__ void step_barrier() {
  static_assert(LATER < 64, "the wait's bits");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"(LATER) : "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (LATER & 15) | (LATER >> 4) << 14);
}

// Fragments of 32 rows x 128 columns. A lane's part is of row lane % 32: pieces 2 h, 2 h + 1, 2 h + 4 and 2 h + 5
// (h = lane / 32), the same for both operands.
struct Raw {
  u32x4_t v[4];
  // where the first piece stands in the fragment's rows of 128 bytes; the others' places are that one ^ piece(i)
  static __device__ __forceinline__ int first(int lane) {
    const int row = lane % 32;
    return row * kBlockK + ((2 * (lane / 32) ^ (row >> 1 & 7)) * 16);
  }
  static constexpr int piece(int i) { return 16 * (i & 1) + 64 * (i >> 1); }
};
// As multiplied: e4m3, or widened to bfloat16
template <bool WIDE>
struct Fragment : Raw {
  __device__ __forceinline__ void take(const Raw& r) { static_cast<Raw&>(*this) = r; }
  __device__ __forceinline__ i32x8_t part(int h) const {
    return __builtin_bit_cast(i32x8_t, __builtin_shufflevector(v[2 * h], v[2 * h + 1], 0, 1, 2, 3, 4, 5, 6, 7));
  }
};
template <>
struct Fragment<true> {
  bf16x8_t v[8];
  __device__ __forceinline__ void take(const Raw& r) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = widen_e4m3(u32x2_t{r.v[i / 2][2 * (i & 1)], r.v[i / 2][2 * (i & 1) + 1]});
  }
};
// The products' sums: token lane % 32, register 4 g + k: row 8 g + 4 (lane / 32) + k
typedef f32x16_t Sum;
__device__ __forceinline__ int first_row(int lane, int g) { return 8 * g + 4 * (lane / 32); }
__device__ __forceinline__ Sum multiply(const Fragment<false>& a, const Fragment<false>& b) {
  Sum p = {};
#pragma unroll
  for (int h = 0; h < 2; ++h) p = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a.part(h), b.part(h), p, 0, 0, 0, 0, 0, 0);
  return p;
}
__device__ __forceinline__ Sum multiply(const Fragment<true>& a, const Fragment<true>& b) {
  Sum p = {};
#pragma unroll
  for (int i = 0; i < 8; ++i) p = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.v[i], b.v[i], p, 0, 0, 0);
  return p;
}

// WR x WT waves, each NR x NT fragments: a workgroup tile of 32 WR NR rows of W x 32 WT NT tokens; STAGES steps' operands in LDS.
template <int WR, int WT, int NR, int NT, int STAGES>
struct Shape {
  static constexpr int kWaves = WR * WT, kThreads = kWaves * kWave, kWaveRows = NR * 32, kWaveTokens = NT * 32;
  static constexpr int kRows = WR * kWaveRows, kTokens = WT * kWaveTokens;
  static constexpr int kStage = (kRows + kTokens) * kBlockK;  // LDS of a step's operands: STAGES of them, then
  static constexpr int kScales = (kRows + kTokens) * 4;       // the scales of twice as many steps, and what nobody reads
  static constexpr int kSlots = STAGES <= 2 ? 4 : 8;
  static constexpr int kScales0 = STAGES * kStage, kSpare = kScales0 + kSlots * kScales, kAll = kSpare + kWaves * 256;
  static constexpr int kPitch = kWaveRows + 4, kEpilogue = kWaves * 32 * kPitch * 4;  // floats of a token's row in the epilogue
  static constexpr int kLds = kAll > kEpilogue ? kAll : kEpilogue;
};

template <int WR, int WT, int NR, int NT, int STAGES, bool WIDE, bool W_ROWS, bool EXPERTS>
__global__ __launch_bounds__(WR * WT * kWave, 2) void fp8_tile_kernel(
    const uint8_t* __restrict__ X, const float* __restrict__ x_scales, const uint8_t* __restrict__ W,
    const float* __restrict__ w_scales, Epilogue ep, void* Y, int past_caches, int M, int K, int n_out, int tiles_n, Groups groups) {
  using S = Shape<WR, WT, NR, NT, STAGES>;
  constexpr int BN = S::kRows, BM = S::kTokens, kWaves = S::kWaves;
  extern __shared__ __align__(1024) uint8_t lds[];  // S::kLds, of which the compiler would take fewer waves for granted
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
  const int wave_n = wave / WT * S::kWaveRows, wave_m = wave % WT * S::kWaveTokens;  // of the tile

  // What a wave loads: pieces of eight rows, a lane 16 bytes of one. Columns past K come as zeros; rows past the last are
  // the last one again, and their results are not stored.
  const int rows_n = min(BN, n_out - n0), rows_m = min(BM, M - m0);
  const uint8_t *const w0 = W + (e * n_out + n0) * K, *const x0 = X + (row0 + m0) * K;
  int l_row = 8 * wave + (lane >> 3);
  const int l_col = ((lane & 7) ^ (4 * (wave & 1) + (lane >> 4))) * 16;
  static_assert(kWaves % 2 == 0, "a wave's pieces are all even or all odd");
  constexpr int kLoadsW = BN / 8 / kWaves, kLoadsX = BM / 8 / kWaves;
  static_assert(BN % (8 * kWaves) == 0 && BM % (8 * kWaves) == 0, "whole pieces");
  constexpr int kX = BN * kBlockK, kScaleW = BM * 4;  // in a step's operands, in its scales
  const float* const w_scale = w_scales + e * KB * (W_ROWS ? n_out : (n_out + 127) / 128);
  // A wave's 64 scales: the tokens', then the rows' of W; one with none loads nothing to a place that nobody reads.
  const bool of_x = wave < BM / 64, of_w = W_ROWS && !of_x && wave < BM / 64 + BN / 64;
  const int scales_first = (of_x ? wave : wave - BM / 64) * 64, scales_end = (of_x ? rows_m : rows_n) * 4;
  const float* const scales0 = of_x ? x_scales + row0 + m0 : w_scale + n0;
  const int64_t scales_step = of_x ? all_rows : n_out;
  const int scales_ring = of_x || of_w ? S::kSlots - 1 : 0;
  const int scales_to = of_x   ? S::kScales0 + scales_first * 4
                        : of_w ? S::kScales0 + kScaleW + scales_first * 4
                               : S::kSpare + wave * 256;
  const int scales_off = of_x || of_w ? (scales_first + lane) * 4 : kAway;
  // Load d of step kb, to a stage. Of a step past the last nothing is read, and zeros are written. No branches, here and in the loop:
  // across them the compiler would move the multiply-adds away from the matrix instructions that they belong to.
  constexpr int kLoads = kLoadsW + kLoadsX + 1;
  auto load = [&](int kb, int stage, int d) __attribute__((always_inline)) {
    if (d == kLoads - 1) {
      const __amdgpu_buffer_rsrc_t rs =
          __builtin_amdgcn_make_buffer_rsrc((void*)(scales0 + kb * scales_step), (short)0, scales_end, kBuffer);
      load_to_lds<4>(rs, lds + scales_to + (kb & scales_ring) * S::kScales, kb < KB ? scales_off : kAway, 0);
    } else {
      const bool of_w = d < kLoadsW;
      const int t = kWaves * (of_w ? d : d - kLoadsW);
      asm("" : "+v"(l_row));  // the rows' offsets are formed here each time: there are no registers to keep them in
      const int rows = of_w ? rows_n : rows_m;
      const __amdgpu_buffer_rsrc_t rs =
          __builtin_amdgcn_make_buffer_rsrc((void*)(of_w ? w0 : x0), (short)0, rows * K, kBuffer);
      load_to_lds<16>(rs, lds + stage * S::kStage + (of_w ? 0 : kX) + (wave + t) * 1024,
                      __umul24(min(l_row + 8 * t, rows - 1), K) + (kb * kBlockK + l_col < K ? l_col : kAway),
                      min(kb, KB - 1) * kBlockK);  // an offset past the descriptor's size could wrap in its bounds check
    }
  };
  static_assert(!W_ROWS || BM / 64 + BN / 64 <= kWaves, "a wave for each 64 scales");

  // A lane's pieces of a fragment. Their places are formed at each read (the asm hides that they are the same), which takes
  // fewer registers than keeping them.
  int at = Raw::first(lane);
  auto read = [&](const uint8_t* rows, Raw& r) __attribute__((always_inline)) {
    asm("" : "+v"(at));
#pragma unroll
    for (int i = 0; i < 4; ++i) r.v[i] = *(const u32x4_t*)(rows + (at ^ Raw::piece(i)));
  };

  // The steps. p of a fragment is added to the sums while the next one's matrix instructions run; the last one's in the next
  // step. A step's last LDS reads lie before its last column of fragments: there the waves meet, the step's place in LDS takes
  // the loads of the step STAGES on, and the next one's first fragments are read as the present ones are done with.
  using F = Fragment<WIDE>;
  constexpr int kBlocks = NR * NT;
  static_assert(NT % 2 == 0, "rings with constant indexes");
  F a[NR], b[2];
  Raw raw;  // WIDE: of the next column of fragments
  Sum acc[NR][NT], p[2];
  float s[2] = {0.0f, 0.0f}, s_next;  // scales of this column's tokens and the last's; the next one's as read
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = Sum{};
  p[0] = p[1] = Sum{};
  const float* const sw_block = w_scale + (size_t)(min(n0 + wave_n, n_out - 1) / 128) * KB;
  const float* const x_scale = (const float*)(lds + S::kScales0) + wave_m + lane % 32;
  const float* const r_scale = (const float*)(lds + S::kScales0 + kScaleW) + wave_n;
  auto read_now = [&](const uint8_t* rows, F& f) __attribute__((always_inline)) {
    if constexpr (WIDE) {
      Raw r;
      read(rows, r);
      f.take(r);
    } else {
      read(rows, f);
    }
  };
  auto add = [&](int kb, auto tt) __attribute__((always_inline)) {  // p of fragment t of step kb
    constexpr int t = decltype(tt)::value, i = t % NR, j = t / NR;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      f32x4_t by = {s[j & 1], s[j & 1], s[j & 1], s[j & 1]};
      if constexpr (W_ROWS) by *= *(const f32x4_t*)(r_scale + (kb & (S::kSlots - 1)) * (S::kScales / 4) + i * 32 + first_row(lane, g));
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][j][4 * g + k] = fmaf(p[t & 1][4 * g + k], by[k], acc[i][j][4 * g + k]);
    }
  };
  // A step's loads are spread over kSpread fragments from its last column on, so that no wave waits with its matrix
  // instructions behind a queue of loads.
  constexpr int kSpread = NR + 1, kEachLoads = (kLoads + kSpread - 1) / kSpread;
  constexpr int kFirst = NR * kEachLoads < kLoads ? NR * kEachLoads : kLoads;  // issued in the step itself
  static_for<STAGES>([&](auto st) __attribute__((always_inline)) {
    constexpr int step = decltype(st)::value;
    static_for<step + 1 < STAGES ? kLoads : kFirst>([&](auto d) __attribute__((always_inline)) { load(step, step, decltype(d)::value); });
  });
  step_barrier<(STAGES - 2) * kLoads + kFirst>();
  float sw = W_ROWS ? 1.0f : sw_block[0];
#pragma unroll
  for (int i = 0; i < NR; ++i) read_now(lds + (wave_n + i * 32) * kBlockK, a[i]);
  read_now(lds + kX + wave_m * kBlockK, b[0]);
  s_next = x_scale[0];
  int now_at = 0, last_at = STAGES - 1;  // stages of this step and the last one
  for (int kb = 0; kb < KB; ++kb) {
    const int next_at = now_at + 1 < STAGES ? now_at + 1 : 0;
    const uint8_t* const x = lds + now_at * S::kStage + kX + wave_m * kBlockK;
    const uint8_t* const next = lds + next_at * S::kStage;  // after the last step: of what lies there
    const float sw_next = W_ROWS ? 1.0f : sw_block[min(kb + 1, KB - 1)];
    static_for<kBlocks>([&](auto tt) __attribute__((always_inline)) {
      constexpr int t = decltype(tt)::value, i = t % NR, j = t / NR;
      if constexpr (i == 0) {
        if constexpr (j + 1 < NT) {
          if constexpr (WIDE) read(x + (j + 1) * 32 * kBlockK, raw);
          else read(x + (j + 1) * 32 * kBlockK, b[(j + 1) & 1]);
        } else {
          step_barrier<(STAGES - 2) * kLoads>();  // the next step's loads have arrived
          if constexpr (WIDE) read(next + kX + wave_m * kBlockK, raw);
          else read(next + kX + wave_m * kBlockK, b[0]);
        }
      }
      constexpr int kTurn = t >= kBlocks - NR ? t - (kBlocks - NR) : t + NR;  // of the spread loads
      constexpr int kFrom = kTurn * kEachLoads;
      constexpr int kCount = kFrom >= kLoads ? 0 : kLoads - kFrom < kEachLoads ? kLoads - kFrom : kEachLoads;
      static_for<kCount>([&](auto d) __attribute__((always_inline)) {
        constexpr bool kNow = t >= kBlocks - NR;
        load(kNow ? kb + STAGES : kb + STAGES - 1, kNow ? now_at : last_at, kFrom + decltype(d)::value);
      });
      if constexpr (i == 0) {
        s[j & 1] = s_next * sw;
        s_next = x_scale[((j + 1 < NT ? kb : kb + 1) & (S::kSlots - 1)) * (S::kScales / 4) + 32 * ((j + 1) % NT)];
      }
      const Sum now = multiply(a[i], b[j & 1]);
      // The first step's first addition, of p = 0, takes step 0's scales: a place that this call has not filled can hold NaN.
      add(t > 0 ? kb : max(kb - 1, 0), std::integral_constant<int, (t + kBlocks - 1) % kBlocks>{});
      p[t & 1] = now;
      if constexpr (WIDE && i == NR - 1) b[(j + 1) & 1].take(raw);
      constexpr int kInstructions = WIDE ? 8 : 2, kEach = WIDE ? 4 : 8;
#pragma unroll
      for (int k = 0; k < kInstructions; ++k) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);      // a matrix instruction
        __builtin_amdgcn_sched_group_barrier(0x002, kEach, 0);  // vector instructions
        if (k < kCount) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);  // a load
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (j == NT - 1) read_now(next + (wave_n + i * 32) * kBlockK, a[i]);
    });
    sw = sw_next;
    last_at = now_at;
    now_at = next_at;
  }
  add(KB - 1, std::integral_constant<int, kBlocks - 1>{});
  // The result through LDS, 32 tokens at a time in a part of each wave's own, so that loads and stores of the epilogue take
  // whole token rows of the wave's outputs. All of a part's loads, then all its sums, then all its stores: no branch between.
  step_barrier<0>();
  constexpr int kLanes = S::kWaveRows / 4, kRound = kWave / kLanes, kRounds = 32 / kRound;
  constexpr bool kBf16 = !WIDE;  // Y's type
  float* const mine = (float*)lds + wave * 32 * S::kPitch;
  const int c = lane % kLanes * 4, n = n0 + wave_n + c, left = n_out - n;
  const bool vec = left >= 4;  // at any alignment (462 rows 3840 -> 2381 with gate and residual: whole call 44.7 -> 32 us)
  const f32x4_t bias = ep.bias && left > 0 ? widen4(load_raw4<true>(ep.bias, e * n_out + n, kBf16, vec, left), kBf16) : f32x4_t{0, 0, 0, 0};
  // whole: every entry of the wave's exists; past: stores that pass the caches
  const auto finish = [&](auto whole, auto past) __attribute__((always_inline)) {
    static_for<NT>([&](auto jj) __attribute__((always_inline)) {
      constexpr int j = decltype(jj)::value;
      u32x4_t gate[kRounds], residual[kRounds];
      f32x4_t y[kRounds];
      const auto place = [&](int r, size_t& at) __attribute__((always_inline)) {  // of a lane's four entries in round r
        const int m = m0 + wave_m + 32 * j + r * kRound + lane / kLanes;
        at = (row0 + m) * n_out + n;
        return decltype(whole)::value || (m < M && left > 0);
      };
      const auto load = [&](const void* p, u32x4_t (&v)[kRounds]) __attribute__((always_inline)) {
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
          size_t at;
          if (place(r, at)) v[r] = load_raw4<true>(p, at, kBf16, decltype(whole)::value || vec, left);
          else v[r] = u32x4_t{0, 0, 0, 0};
        }
      };
      if (ep.gate) load(ep.gate, gate);
      if (ep.residual) load(ep.residual, residual);
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const Sum& v = acc[i][j];
          *(f32x4_t*)(mine + lane % 32 * S::kPitch + i * 32 + first_row(lane, g)) =
              f32x4_t{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int r = 0; r < kRounds; ++r) y[r] = *(const f32x4_t*)(mine + (r * kRound + lane / kLanes) * S::kPitch + c) + bias;
      with_activation(ep.act, [&](auto act) __attribute__((always_inline)) {
#pragma unroll
        for (int r = 0; r < kRounds; ++r) y[r] = activate4<decltype(act)::value>(y[r]);
      });
      if (ep.gate) {
#pragma unroll
        for (int r = 0; r < kRounds; ++r) y[r] *= widen4(gate[r], kBf16);
      }
      if (ep.residual) {
#pragma unroll
        for (int r = 0; r < kRounds; ++r) y[r] += widen4(residual[r], kBf16);
      }
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        size_t at;
        if (place(r, at)) store4<decltype(past)::value, true>(Y, at, kBf16, decltype(whole)::value || vec, left, y[r]);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    });
  };
  // A Y too large for the caches goes past them: the rows of X and W that later tiles read stay there instead.
  if (n0 + wave_n + S::kWaveRows > n_out || m0 + wave_m + S::kWaveTokens > M) finish(std::false_type{}, std::false_type{});
  else if (past_caches) finish(std::true_type{}, std::true_type{});
  else finish(std::true_type{}, std::false_type{});
}

int64_t tile_blocks(const Fp8Call& c, int tokens) {
  return c.offsets ? most_group_tiles(c.M, c.experts, tokens) : ceil_div(c.M, tokens);
}

template <int WR, int WT, int NR, int NT, int STAGES, bool WIDE, bool W_ROWS>
hipError_t launch_shape(const Fp8Call& c, hipStream_t stream) {
  using S = Shape<WR, WT, NR, NT, STAGES>;
  const int tiles_n = (int)ceil_div(c.n_out, S::kRows);
  const dim3 grid((unsigned)(8 * ceil_div(tiles_n * tile_blocks(c, S::kTokens), 8)));
  const Groups groups{c.offsets, (int)c.experts, (int)c.M};
  const int past = (double)c.M * c.n_out * (WIDE ? 4 : 2) > kNonTemporalYBytes;
  const auto kernel = c.offsets ? fp8_tile_kernel<WR, WT, NR, NT, STAGES, WIDE, W_ROWS, true> : fp8_tile_kernel<WR, WT, NR, NT, STAGES, WIDE, W_ROWS, false>;
  kernel<<<grid, dim3(S::kThreads), S::kLds, stream>>>((const uint8_t*)c.X, c.x_scales, c.W, c.w_scales, c.ep, c.Y,
                                                 past, (int)c.M, (int)c.n_in, (int)c.n_out, tiles_n, groups);
  return hipGetLastError();
}

}  // namespace

bool fp8_tile_grid_fits(const Fp8Call& c, int rows, int tokens) {
  return tile_blocks(c, tokens) * ceil_div(c.n_out, rows) < (int64_t(1) << 23);
}

hipError_t launch_fp8_tile(const Fp8Call& c, int rows, int stages, hipStream_t stream) {
  if (rows == 256) return launch_shape<4, 2, 2, 4, 2, false, false>(c, stream);
  const auto launch = [&](auto st) {
    constexpr int kStages = decltype(st)::value;
    if (!c.y_bf16) return c.w_rows ? launch_shape<2, 2, 2, 2, kStages, true, true>(c, stream) : launch_shape<2, 2, 2, 2, kStages, true, false>(c, stream);
    return c.w_rows ? launch_shape<2, 2, 2, 2, kStages, false, true>(c, stream) : launch_shape<2, 2, 2, 2, kStages, false, false>(c, stream);
  };
  return stages == 2 ? launch(std::integral_constant<int, 2>{}) : launch(std::integral_constant<int, 4>{});
}

}  // namespace splr
