// The 8-bit product for few tokens: a workgroup has 16 NT tokens and several tiles of 16 rows of W, one after the other, its
// waves the blocks of 128 columns in turn.
//
//   acc[n][m] += sx[m][kb] sw[n][kb] sum over k in block kb of W[n][k] X[m][k]
//
// Reading W bounds this kernel. Each wave has a ring of its own in LDS, AHEAD blocks deep, that loads fill without registers
// between and without barriers, from one tile into the next: whole lines of 128 bytes of eight rows at a time (one row 14336 ->
// 4096: 15.2 us; with fragments read to registers, 64 bytes of 16 rows at a time, 17.7). Both operands become bfloat16 in
// registers (exact), so that the sums over a block are float32 sums on the bfloat16 matrix cores, whose time does not show here.
// X that is not held in 8 bits yet is quantised by the workgroup, into LDS, while the first of W arrives: a launch of its own
// would cost more than the few rows that a tile has.
#include "fp8.hpp"
#include "tile_common.hpp"

namespace splr {
namespace {

constexpr int kFewWaves = 8, kFewThreads = kFewWaves * kWave;
constexpr int kBuffer = 0x00020000;  // word 3 of a raw buffer descriptor: plain byte-addressed loads
constexpr int kAway = 1 << 30;       // past every descriptor's end: such a load gives zeros
constexpr int kFragment = 16 * kBlockK;
enum : int { kXe4m3 = 0, kXbf16 = 1, kXf32 = 2 };

// Dynamic LDS: the waves' rings (a block's fragment of W and a place for 64 of its scales; with X in e4m3 its fragments and
// scales too), then, of X that the workgroup quantises, rows of KB blocks, 16 bytes apart from a multiple of the banks, and the scales [KB][rows]
__host__ __device__ constexpr int slot_bytes(int NT, bool e4m3) {
  return kFragment + 256 + (e4m3 ? kFragment * NT + 256 : 0);
}
__host__ __device__ constexpr int x_pitch(int KB) { return KB * kBlockK + 16; }
__host__ __device__ constexpr int x_bytes(int rows, int KB) { return rows * (x_pitch(KB) + 4 * KB); }

// All of this wave's loads but the last LATER have arrived. The builtin tells the compiler.
template <int LATER>
__device__ __forceinline__ void wait_loads() {
  static_assert(LATER < 64, "");
  asm volatile("s_waitcnt vmcnt(%0)" ::"i"(LATER) : "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (LATER & 15) | (LATER >> 4) << 14);
}
__device__ __forceinline__ void to_lds16(__amdgpu_buffer_rsrc_t rs, uint8_t* lds, int offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)lds, 16, offset, 0, 0, 0);
}

template <int NT, int AHEAD, int XT, bool EXPERTS>
__global__ __launch_bounds__(kFewThreads) void fp8_few_kernel(
    const void* __restrict__ X, const float* __restrict__ x_scales, const uint8_t* __restrict__ W,
    const float* __restrict__ w_scales, int w_rows, Epilogue ep, void* Y, int y_bf16, int M, int K, int n_out, int tiles,
    int cap, Groups groups) {
  constexpr int kPitch = 20;  // floats of a token's 16 sums in LDS
  constexpr bool kHeld = XT == kXe4m3;
  constexpr int kSlot = slot_bytes(NT, kHeld), kLoads = 3 + (kHeld ? 2 * NT + 1 : 0);  // of a block
  constexpr int kScaleW = kFragment, kX = kFragment + 256, kScaleX = kX + kFragment * NT;  // in a slot
  __shared__ __align__(16) float sums[2][kFewWaves][NT][16 * kPitch];
  extern __shared__ __align__(1024) uint8_t lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = lane & 15, quad = lane >> 4;
  const int KB = (K + kBlockK - 1) / kBlockK;
  size_t e = 0, row0 = 0;
  int rows = M, m0 = blockIdx.y * 16 * NT;
  if constexpr (EXPERTS) {
    const GroupTile gt = find_group_tile<16 * NT>(groups, blockIdx.y);
    if (gt.expert < 0) return;
    e = gt.expert;
    row0 = gt.lo;
    rows = gt.rows;
    m0 = (blockIdx.y - gt.first) * 16 * NT;
  }
  const int here = min(16 * NT, rows - m0);  // rows past the last repeat it and are not stored
  const __amdgpu_buffer_rsrc_t xrs =
      __builtin_amdgcn_make_buffer_rsrc((void*)((const uint8_t*)X + (row0 + m0) * K), (short)0, here * K, kBuffer);
  const float* const ws = w_scales + e * KB * (w_rows ? n_out : (n_out + 127) / 128);

  // A load's lanes: row lane / 8 of eight, 16 bytes; piece c of row r goes to place c ^ (r / 2 % 8) of its 128 bytes
  uint8_t* const ring = lds + wave * AHEAD * kSlot;
  const int l_row = lane >> 3;
  const auto to_lds4 = [&](const float* from, int n, uint8_t* to) __attribute__((always_inline)) {  // entry n - 1 again past it
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)from, (short)0, n * 4, kBuffer);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (__attribute__((address_space(3))) void*)to, 4, min(lane, n - 1) * 4, 0, 0, 0);
  };
  const auto load = [&](int tile, int kb, int slot) __attribute__((always_inline)) {
    uint8_t* const to = ring + slot * kSlot;
    const int n0 = min(tile, tiles - 1) * 16, n_here = min(16, n_out - n0), end = tile < tiles ? K : 0;
    const __amdgpu_buffer_rsrc_t wrs =
        __builtin_amdgcn_make_buffer_rsrc((void*)(W + (e * n_out + n0) * K), (short)0, n_here * K, kBuffer);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = kb * kBlockK + ((lane & 7) ^ (4 * h + (lane >> 4))) * 16, col = c < end ? c : kAway;
      to_lds16(wrs, to + 1024 * h, min(8 * h + l_row, n_here - 1) * K + col);
      if constexpr (kHeld) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
          to_lds16(xrs, to + kX + kFragment * j + 1024 * h, min(16 * j + 8 * h + l_row, here - 1) * K + col);
      }
    }
    const int b = min(kb, KB - 1);  // of a block or tile past the last, W and X are zeros
    to_lds4(w_rows ? ws + (size_t)b * n_out + n0 : ws + (size_t)(n0 / 128) * KB + b, w_rows ? n_here : 1, to + kScaleW);
    if constexpr (kHeld) to_lds4(x_scales + (size_t)b * M + row0 + m0, here, to + kScaleX);
  };
  // the block that is loaded next
  const int turns = (KB + kFewWaves - 1) / kFewWaves, stride = gridDim.x;
  int next_tile = blockIdx.x, next_turn = 0;
  const auto load_next = [&](int slot) __attribute__((always_inline)) {
    load(next_tile, next_turn * kFewWaves + wave, slot);
    const bool more = next_turn + 1 < turns;
    next_turn = more ? next_turn + 1 : 0;
    next_tile = more ? next_tile : next_tile + stride;
  };
  // X: 16 lanes a block, eight entries a lane. The first rounds' are asked for before W, behind which they would arrive.
  uint8_t* const xq = lds + kFewWaves * AHEAD * kSlot;
  float* const xs = (float*)(xq + cap * x_pitch(KB));
  const int x_blocks = here * KB;
  struct Place {
    int t, kb, col;
    bool exists;
  };
  const auto x_place = [&](int round) __attribute__((always_inline)) {
    const int i = (round * kFewWaves + wave) * 4 + (lane >> 4), t = min(i / KB, here - 1), kb = i - i / KB * KB;
    return Place{t, kb, kb * kBlockK + 8 * (lane & 15), i < x_blocks};
  };
  const auto x_load = [&](int round, float (&v)[8]) __attribute__((always_inline)) {
    const Place p = x_place(round);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (p.exists && p.col < K) load8<XT == kXbf16>(X, (row0 + m0 + p.t) * K + p.col, v);
  };
  const auto x_store = [&](int round, float (&v)[8]) __attribute__((always_inline)) {
    const Place p = x_place(round);
    uint32_t most = largest_bits(v);
    if (__any(most >= kInfBits)) most = drop_infinite(v);
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) most = max(most, (uint32_t)__shfl_xor((int)most, off));
    const float s = block_scale(__uint_as_float(most)), inv = 1.0f / s;
    if (p.exists) {
      *(u32x2_t*)(xq + p.t * x_pitch(KB) + p.col) = u32x2_t{to_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                                                            to_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv)};
      if ((lane & 15) == 0) xs[p.kb * cap + p.t] = s;
    }
  };
  constexpr int kRounds = 4;
  float v[kHeld ? 1 : kRounds][8];
  if constexpr (!kHeld) {
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
      if (r * kFewWaves * 4 < x_blocks) x_load(r, v[r]);
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) load_next(u);
  if constexpr (!kHeld) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
      if (r * kFewWaves * 4 < x_blocks) x_store(r, v[r]);
    for (int r = kRounds; r * kFewWaves * 4 < x_blocks; ++r) {
      x_load(r, v[0]);
      x_store(r, v[0]);
    }
    lds_barrier();
  }

  // A fragment: a lane has row (token) lane % 16, pieces quad and quad + 4
  const int place = sub * kBlockK + ((quad ^ (sub >> 1)) * 16);
  int token[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) token[j] = min(16 * j + sub, here - 1);
  f32x4_t acc[NT];
  int slot = 0, turn_of_sums = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += stride) {
    // the epilogue's operands first: one wave finishes a fragment, another one in the next tile
    const int n0 = tile * 16, out_row = n0 + 4 * quad, left = n_out - out_row;
    const int mine = (wave - turn_of_sums * NT) & (kFewWaves - 1);
    const bool finishes = mine < NT && m0 + 16 * mine + sub < rows && left > 0, vec = left >= 4;
    const size_t at = (row0 + m0 + 16 * mine + sub) * n_out + out_row;
    u32x4_t bias = {0, 0, 0, 0}, gate = bias, residual = bias;
    if (finishes) {
      if (ep.bias) bias = load_raw4<true>(ep.bias, e * n_out + out_row, y_bf16, vec, left);
      if (ep.gate) gate = load_raw4<true>(ep.gate, at, y_bf16, vec, left);
      if (ep.residual) residual = load_raw4<true>(ep.residual, at, y_bf16, vec, left);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j] = f32x4_t{0, 0, 0, 0};
    for (int turn = 0; turn < turns; ++turn) {
      wait_loads<(AHEAD - 1) * kLoads>();
      const uint8_t* const from = ring + slot * kSlot;
      const int kb = min(turn * kFewWaves + wave, KB - 1);
      u32x4_t w[2], x[NT][2];
      float s[NT];
#pragma unroll
      for (int h = 0; h < 2; ++h) w[h] = *(const u32x4_t*)(from + (place ^ (64 * h)));
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (kHeld) {
#pragma unroll
          for (int h = 0; h < 2; ++h) x[j][h] = *(const u32x4_t*)(from + kX + kFragment * j + (place ^ (64 * h)));
          s[j] = ((const float*)(from + kScaleX))[token[j]];
        } else {
          const uint8_t* const p = xq + token[j] * x_pitch(KB) + kb * kBlockK + 16 * quad;
          x[j][0] = *(const u32x4_t*)p;
          x[j][1] = *(const u32x4_t*)(p + 64);
          s[j] = xs[kb * cap + token[j]];
        }
      }
      const f32x4_t by = *(const f32x4_t*)(from + kScaleW + 16 * quad);
      __builtin_amdgcn_s_waitcnt(0xC07F);  // the fragments are in registers, so their place may be filled again
      __builtin_amdgcn_sched_barrier(0);
      load_next(slot);
      __builtin_amdgcn_sched_barrier(0);
      slot = slot + 1 < AHEAD ? slot + 1 : 0;
      if (turn * kFewWaves + wave >= KB) continue;
      bf16x8_t wide[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) wide[i] = widen_e4m3(u32x2_t{w[i / 2][2 * (i & 1)], w[i / 2][2 * (i & 1) + 1]});
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        f32x4_t p = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          p = mfma16x16x32(wide[i], widen_e4m3(u32x2_t{x[j][i / 2][2 * (i & 1)], x[j][i / 2][2 * (i & 1) + 1]}), p);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[j][k] = fmaf(p[k], s[j] * by[k], acc[j][k]);
      }
    }
    // D fragment: token lane % 16, rows 4 (lane / 16) .. +3; the waves' sums in their order. Two places for them in turn, so
    // that one barrier a tile is enough.
    float(*const parts)[NT][16 * kPitch] = sums[turn_of_sums & 1];
#pragma unroll
    for (int j = 0; j < NT; ++j) *(f32x4_t*)&parts[wave][j][sub * kPitch + 4 * quad] = acc[j];
    lds_barrier();
    if (finishes) {
      f32x4_t sum = *(const f32x4_t*)&parts[0][mine][sub * kPitch + 4 * quad];
#pragma unroll
      for (int v = 1; v < kFewWaves; ++v) sum += *(const f32x4_t*)&parts[v][mine][sub * kPitch + 4 * quad];
      store4<false, true>(Y, at, y_bf16, vec, left, finish4(sum, widen4(bias, y_bf16), ep, widen4(gate, y_bf16), widen4(residual, y_bf16)));
    }
    ++turn_of_sums;
  }
  wait_loads<0>();  // nothing is written to LDS after the workgroup's end
}

int64_t few_blocks(const Fp8Call& c, int tokens) { return c.offsets ? most_group_tiles(c.M, c.experts, tokens) : ceil_div(c.M, tokens); }
int few_cap(const Fp8Call& c, int tokens) { return (int)(c.M < tokens ? c.M : tokens); }
// Blocks in a ring: as many as LDS has room for, two where a wave has no more
constexpr int most_ahead(int tokens, bool e4m3) { return !e4m3 ? 4 : tokens == 16 ? 3 : 2; }
bool short_ring(const Fp8Call& c) { return ceil_div(c.n_in, kBlockK) <= 2 * kFewWaves; }
int few_lds(const Fp8Call& c, int tokens, bool e4m3) {
  return kFewWaves * (short_ring(c) ? 2 : most_ahead(tokens, e4m3)) * slot_bytes(tokens / 16, e4m3) +
         (e4m3 ? 0 : x_bytes(few_cap(c, tokens), (int)ceil_div(c.n_in, kBlockK)));
}

constexpr int kLdsBytes = 160 << 10;  // of a CU
constexpr int kSumsBytes(int tokens) { return 2 * kFewWaves * tokens * 20 * 4; }
// As many workgroups as the chip holds at once, each with a share of the row tiles
dim3 few_grid(const Fp8Call& c, int tokens) {
  const int64_t tiles = ceil_div(c.n_out, 16), blocks = few_blocks(c, tokens);
  const int64_t at_once = 256 * (2 * (few_lds(c, tokens, c.x_type == 2) + kSumsBytes(tokens)) <= kLdsBytes ? 2 : 1);
  const int64_t share = ceil_div(tiles * blocks, at_once);
  return dim3((unsigned)ceil_div(tiles, share < tiles ? share : tiles), (unsigned)blocks);
}

template <int NT, int XT>
hipError_t launch_type(const Fp8Call& c, hipStream_t stream) {
  constexpr int kMost = most_ahead(16 * NT, XT == kXe4m3);
  const Groups groups{c.offsets, (int)c.experts, (int)c.M};
  const auto kernel = c.offsets ? (short_ring(c) ? fp8_few_kernel<NT, 2, XT, true> : fp8_few_kernel<NT, kMost, XT, true>)
                                : (short_ring(c) ? fp8_few_kernel<NT, 2, XT, false> : fp8_few_kernel<NT, kMost, XT, false>);
  kernel<<<few_grid(c, 16 * NT), dim3(kFewThreads), few_lds(c, 16 * NT, XT == kXe4m3), stream>>>(
      c.X, c.x_scales, c.W, c.w_scales, c.w_rows, c.ep, c.Y, c.y_bf16, (int)c.M, (int)c.n_in, (int)c.n_out,
      (int)ceil_div(c.n_out, 16), few_cap(c, 16 * NT), groups);
  return hipGetLastError();
}
template <int NT>
hipError_t launch_tokens(const Fp8Call& c, hipStream_t stream) {
  return c.x_type == 2 ? launch_type<NT, kXe4m3>(c, stream) : c.x_type == 1 ? launch_type<NT, kXbf16>(c, stream) : launch_type<NT, kXf32>(c, stream);
}

}  // namespace

bool fp8_few_grid_fits(const Fp8Call& c, int tokens) { return grid_fits(few_grid(c, tokens), kFewThreads); }
bool fp8_few_quantizes(const Fp8Call& c, int tokens) { return few_lds(c, tokens, false) + kSumsBytes(tokens) <= kLdsBytes; }
hipError_t launch_fp8_few(const Fp8Call& c, int tokens, hipStream_t stream) {
  return tokens == 32 ? launch_tokens<2>(c, stream) : launch_tokens<1>(c, stream);
}

}  // namespace splr
