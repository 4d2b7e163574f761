// Quantisation to e4m3 with a scale for each block (splr_fp8_quantize): s = max(largest finite magnitude / 448, 2^-126),
// entries e4m3(x (1 / s)). Blocks of 1 x 128 or 128 x 128, the result in rows or transposed.
#include "fp8.hpp"

namespace splr {
namespace {

// Blocks of 1 x 128, not transposed: 16 lanes a block, eight entries a lane, one wave four blocks of a row.
template <bool BF16>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const void* __restrict__ X, int64_t rows, int cols,
                                                            uint8_t* __restrict__ Q, float* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const int64_t row = blockIdx.x * (int64_t)4 + (threadIdx.x >> 6);  // a workgroup's scales lie next to each other
  const int kb = blockIdx.y * 4 + lane / 16, col = kb * kBlockK + 8 * (lane & 15);
  if (row >= rows) return;
  float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  const bool here = col < cols;
  if (here) load8<BF16>(X, row * cols + col, v);
  uint32_t m = largest_bits(v);
  if (__any(m >= kInfBits)) m = drop_infinite(v);
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off));
  const float s = block_scale(__uint_as_float(m)), inv = 1.0f / s;
  if (here) {
    u32x2_t q;
    q[0] = to_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
    q[1] = to_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv);
    *(u32x2_t*)(Q + row * cols + col) = q;
    if ((lane & 15) == 0) scales[(size_t)kb * rows + row] = s;
  }
}

// The rest: one workgroup a tile of 128 x 128, a thread two columns (64 apart) of 32 rows. Bound by its narrow accesses, entry
// by entry from X, to Q one byte at a time or, transposed, 16 bytes of 64 rows: bfloat16 in blocks of 128 x 128 4096 x 4096
// 18.7 us (2.7 TB/s; transposed 16.4), 14336 x 4096 60.9 (56.1); of 1 x 128 transposed 2048 x 4096 9.0. The tiles are numbered row after row in
// the grid's x: its y ends at 65535, and there may be 2^17 tiles in either direction.
// TRANSPOSED: Q [cols][pitch], pitch = rows rounded up to 32, zeros past the rows. BLOCK: one scale for the tile.
template <bool BF16, bool TRANSPOSED, bool BLOCK>
__global__ __launch_bounds__(256) void quantize_tile_kernel(const void* __restrict__ X, int64_t rows, int64_t cols,
                                                            int64_t pitch, uint8_t* __restrict__ Q,
                                                            float* __restrict__ scales) {
  __shared__ uint32_t largest[4][128];
  const int c = threadIdx.x & 63, g = threadIdx.x >> 6;
  const unsigned row_tiles = (unsigned)((rows + 127) / 128), col_tiles = (unsigned)((cols + 127) / 128);
  const unsigned row_tile = blockIdx.x / col_tiles, col_tile = blockIdx.x - row_tile * col_tiles;
  const int64_t r0 = row_tile * (int64_t)128, c0 = col_tile * (int64_t)128, row0 = r0 + 32 * g;
  float v[2][32];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t col = c0 + 64 * h + c;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const bool here = col < cols && row0 + i < rows;
      const size_t at = here ? (size_t)((row0 + i) * cols + col) : 0;
      const float x = BF16 ? bf16_bits_to_float(((const uint16_t*)X)[at]) : ((const float*)X)[at];
      v[h][i] = here ? x : 0.0f;
    }
    uint32_t m = largest_bits(v[h]);
    if (m >= kInfBits) m = drop_infinite(v[h]);
    largest[g][64 * h + c] = m;
  }
  __syncthreads();
  uint32_t m[2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
    m[h] = max(max(largest[0][64 * h + c], largest[1][64 * h + c]), max(largest[2][64 * h + c], largest[3][64 * h + c]));
  if constexpr (BLOCK) {
    uint32_t all = max(m[0], m[1]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) all = max(all, (uint32_t)__shfl_xor((int)all, off));
    m[0] = m[1] = all;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t col = c0 + 64 * h + c;
    if (col >= cols) continue;
    const float s = block_scale(__uint_as_float(m[h])), inv = 1.0f / s;
    if constexpr (BLOCK) {
      if (threadIdx.x == 0 && h == 0)
        scales[TRANSPOSED ? (size_t)col_tile * row_tiles + row_tile : (size_t)row_tile * col_tiles + col_tile] = s;
    } else {
      if (g == 0) scales[(size_t)row_tile * cols + col] = s;
    }
    if constexpr (TRANSPOSED) {
      if (row0 >= pitch) continue;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        u32x4_t q;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float* x = v[h] + 16 * p + 4 * i;
          q[i] = to_e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
        }
        *(u32x4_t*)(Q + (size_t)col * pitch + row0 + 16 * p) = q;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (row0 + i < rows) Q[(size_t)(row0 + i) * cols + col] = (uint8_t)to_e4m3x2<false>(v[h][i] * inv, 0.0f, 0);
    }
  }
}

dim3 rows_grid(int64_t rows, int64_t cols) {
  return dim3((unsigned)ceil_div(rows, 4), (unsigned)ceil_div(cols, 4 * kBlockK));
}
dim3 tile_grid(int64_t rows, int64_t cols) { return dim3((unsigned)(ceil_div(cols, 128) * ceil_div(rows, 128))); }

}  // namespace

bool fp8_quantize_grids_fit(int64_t rows, int64_t cols, bool block, bool transposed) {
  return grid_fits(block || transposed ? tile_grid(rows, cols) : rows_grid(rows, cols), 256);
}

hipError_t launch_fp8_quantize(const void* X, int64_t rows, int64_t cols, bool bf16, bool block, bool transposed, void* Q,
                               float* scales, hipStream_t stream) {
  if (!block && !transposed) {
    const auto kernel = bf16 ? quantize_rows_kernel<true> : quantize_rows_kernel<false>;
    kernel<<<rows_grid(rows, cols), dim3(256), 0, stream>>>(X, rows, (int)cols, (uint8_t*)Q, scales);
    return hipGetLastError();
  }
  const auto launch = [&](auto kernel) {
    kernel<<<tile_grid(rows, cols), dim3(256), 0, stream>>>(X, rows, cols, ceil_div(rows, 32) * 32, (uint8_t*)Q, scales);
  };
  if (bf16) launch(!transposed ? quantize_tile_kernel<true, false, true> : block ? quantize_tile_kernel<true, true, true> : quantize_tile_kernel<true, true, false>);
  else launch(!transposed ? quantize_tile_kernel<false, false, true> : block ? quantize_tile_kernel<false, true, true> : quantize_tile_kernel<false, true, false>);
  return hipGetLastError();
}

}  // namespace splr
