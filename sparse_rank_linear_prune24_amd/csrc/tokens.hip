// The way of tokens to their experts and back (splr_tokens_*): a stable counting sort of the tokens' slots by expert,
// rows copied to their places, results weighted and added back, and the gradient of that.
//
//   offsets[e] = slots with an id below e      positions[t][j] = offsets[id] + earlier slots with the same id
//   gather     Xs[positions[t][j]] = X[t]      combine  Y[t] = residual[t] + sum_j w[t][j] Z[positions[t][j]]
//   backward   dZ[positions[t][j]] = w[t][j] dY[t],  dw[t][j] = <dY[t], Z[positions[t][j]]>
//
// Sums are float32 in a fixed order; nothing depends on the order in which workgroups run.
#include "common.hpp"
#include "epilogue.hpp"
#include "kernels.hpp"
#include "tokens.hpp"

namespace splr {
namespace {

constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / kWave;

// A slot's expert, -1 when its id names none.
__device__ __forceinline__ int expert_of(const void* ids, int wide, int64_t i, int experts) {
  const int64_t id = wide ? ((const int64_t*)ids)[i] : ((const int32_t*)ids)[i];
  return id >= 0 && id < experts ? (int)id : -1;
}

// counts[e] += slots first .. last-1 with id e, by all threads (integer sums: their order does not matter)
__device__ __forceinline__ void count_slots(const void* ids, int wide, int64_t first, int64_t last, int experts, int* counts,
                                            int tid, int threads) {
  for (int64_t i = first + tid; i < last; i += threads) {
    const int e = expert_of(ids, wide, i, experts);
    if (e >= 0) atomicAdd(counts + e, 1);
  }
}

// Counts of each segment of `segment` slots, [segments][experts].
__global__ __launch_bounds__(kSortThreads) void count_kernel(const void* __restrict__ ids, int wide, int64_t N, int64_t segment,
                                                             int experts, int* __restrict__ counts) {
  extern __shared__ int lds[];
  for (int e = threadIdx.x; e < experts; e += kSortThreads) lds[e] = 0;
  __syncthreads();
  const int64_t first = blockIdx.x * segment;
  count_slots(ids, wide, first, min(first + segment, N), experts, lds, threadIdx.x, kSortThreads);
  __syncthreads();
  for (int e = threadIdx.x; e < experts; e += kSortThreads) counts[(size_t)blockIdx.x * experts + e] = lds[e];
}

// Exclusive prefix sum over the workgroup's threads, thread after thread.
__device__ __forceinline__ int prefix_of_block(int v, int* sums) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int upto = v;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(upto, off);
    if (lane >= off) upto += o;
  }
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < wave; ++w) before += sums[w];
  return before + upto - v;
}

// Positions of one segment of slots a workgroup, and the offsets. counts: every segment's counts; NULL: each workgroup
// counts all N slots itself, which saves the first launch where N is small.
__global__ __launch_bounds__(kSortThreads) void place_kernel(const void* __restrict__ ids, int wide, int64_t N, int64_t segment,
                                                             int experts, const int* __restrict__ counts,
                                                             int32_t* __restrict__ offsets, int32_t* __restrict__ positions) {
  extern __shared__ int lds[];
  __shared__ int sums[kSortWaves];
  int* const next = lds;                          // [waves][experts]: where a wave's next slot of an expert goes
  int* const before = lds + kSortWaves * experts;  // slots of the segments before
  int* const total = before + experts;             // all slots
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t first = blockIdx.x * segment, last = min(first + segment, N);
  for (int i = tid; i < (kSortWaves + 2) * experts; i += kSortThreads) lds[i] = 0;
  __syncthreads();
  // each wave's part of the segment: whole groups of 64 slots
  const int64_t part = ceil_div(ceil_div(segment, kSortWaves), 64) * 64;
  const int64_t w_first = min(first + wave * part, last), w_last = min(w_first + part, last);
  count_slots(ids, wide, w_first, w_last, experts, next + wave * experts, lane, kWave);
  if (counts) {
    const int segments = (int)gridDim.x;
    for (int e = tid; e < experts; e += kSortThreads) {
      int b = 0, all = 0;
      for (int s = 0; s < segments; ++s) {
        const int c = counts[(size_t)s * experts + e];
        b += s < (int)blockIdx.x ? c : 0;
        all += c;
      }
      before[e] = b;
      total[e] = all;
    }
  } else {
    count_slots(ids, wide, 0, first, experts, before, tid, kSortThreads);
    count_slots(ids, wide, 0, N, experts, total, tid, kSortThreads);
  }
  __syncthreads();
  const int mine = tid < experts ? total[tid] : 0;
  const int start = prefix_of_block(mine, sums);
  if (tid < experts) {
    if (blockIdx.x == 0) {
      offsets[tid] = start;
      if (tid == experts - 1) offsets[experts] = start + mine;
    }
    int at = start + before[tid];
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = next[w * experts + tid];
      next[w * experts + tid] = at;
      at += c;
    }
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz(experts | 1);
  int* const mine_next = next + wave * experts;
  for (int64_t i0 = w_first; i0 < w_last; i0 += kWave) {
    const int64_t i = i0 + lane;
    const int e = i < w_last ? expert_of(ids, wide, i, experts) : -1;
    // lanes with this lane's expert
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t set = __ballot((e >> b) & 1);
      same &= ((e >> b) & 1) ? set : ~set;
    }
    int at = -1;
    const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
    if (e >= 0) at = mine_next[e] + rank;
    // every lane has read before one of each expert writes, and that before the next round's reads
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (e >= 0 && rank == 0) mine_next[e] = at + __popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (i < w_last) positions[i] = at;
  }
}

// ------------------------------------------------------------------------------------------------- rows

// A row's 16-byte pieces (V = u32x4_t), or its entries where rows are not a multiple of 16 bytes (V: uint8_t, uint16_t,
// uint32_t). One workgroup a token and up to four times 64 V of its row.
template <typename V>
__global__ __launch_bounds__(256) void gather_kernel(const V* __restrict__ X, int row_v, const int32_t* __restrict__ positions,
                                                     int slots, V* __restrict__ Xs, int64_t rows) {
  const int64_t t = blockIdx.x;
  const int c = blockIdx.y * blockDim.x + threadIdx.x;
  if (c >= row_v) return;
  const V v = X[t * row_v + c];
  for (int j = 0; j < slots; ++j) {
    const int64_t p = positions[t * slots + j];
    if (p >= 0 && p < rows) Xs[p * row_v + c] = v;
  }
}

// Eight bfloat16 or four float32 entries as loaded, or one entry (rows that are not a multiple of 16 bytes).
template <bool BF16, bool VEC>
struct Piece {
  static constexpr int kN = !VEC ? 1 : BF16 ? 8 : 4;
  float v[kN];
  __device__ __forceinline__ void load(const void* p, int64_t at) {  // at: in pieces
    if constexpr (!VEC) {
      v[0] = BF16 ? bf16_bits_to_float(((const uint16_t*)p)[at]) : ((const float*)p)[at];
    } else {
      const u32x4_t w = ((const u32x4_t*)p)[at];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
          v[2 * i] = __uint_as_float(w[i] << 16);
          v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
          v[i] = __uint_as_float(w[i]);
        }
      }
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t at) const {
    if constexpr (!VEC) {
      if constexpr (BF16) ((uint16_t*)p)[at] = (uint16_t)round_bf16x2(v[0], v[0]);
      else ((float*)p)[at] = v[0];
    } else {
      u32x4_t w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) w[i] = round_bf16x2(v[2 * i], v[2 * i + 1]);
        else w[i] = __float_as_uint(v[i]);
      }
      ((u32x4_t*)p)[at] = w;
    }
  }
};

// Up to four slots of a token (wave-uniform): row, -1 for none, and weight. Their rows are asked for together.
constexpr int kSlotsAtOnce = 4;
struct Slots4 {
  int64_t p[kSlotsAtOnce];
  float w[kSlotsAtOnce];
  __device__ __forceinline__ void load(const int32_t* positions, const float* weights, int64_t at, int left, int64_t rows) {
#pragma unroll
    for (int j = 0; j < kSlotsAtOnce; ++j) {
      p[j] = j < left ? positions[at + j] : -1;
      if (p[j] >= rows) p[j] = -1;
      w[j] = weights && j < left ? weights[at + j] : 1.0f;
    }
  }
};

template <bool BF16, bool VEC>
__global__ __launch_bounds__(256) void combine_kernel(const void* __restrict__ Z, int64_t rows, int row_v,
                                                      const int32_t* __restrict__ positions, int slots,
                                                      const float* __restrict__ weights, const void* residual, void* Y) {
  using P = Piece<BF16, VEC>;
  const int64_t t = blockIdx.x;
  const int c = blockIdx.y * blockDim.x + threadIdx.x;
  if (c >= row_v) return;
  P sum;
#pragma unroll
  for (int i = 0; i < P::kN; ++i) sum.v[i] = 0.0f;
  for (int j0 = 0; j0 < slots; j0 += kSlotsAtOnce) {
    Slots4 s;
    s.load(positions, weights, t * slots + j0, slots - j0, rows);
    P z[kSlotsAtOnce];
#pragma unroll
    for (int j = 0; j < kSlotsAtOnce; ++j)
      if (s.p[j] >= 0) z[j].load(Z, s.p[j] * row_v + c);
#pragma unroll
    for (int j = 0; j < kSlotsAtOnce; ++j)
      if (s.p[j] >= 0) {
#pragma unroll
        for (int i = 0; i < P::kN; ++i) sum.v[i] = fmaf(s.w[j], z[j].v[i], sum.v[i]);
      }
  }
  if (residual) {
    P r;
    r.load(residual, t * row_v + c);
#pragma unroll
    for (int i = 0; i < P::kN; ++i) sum.v[i] += r.v[i];
  }
  sum.store(Y, t * row_v + c);
}

// One workgroup a token: dY's row is read once for every four slots (from L1 after the first).
template <bool BF16, bool VEC>
__global__ __launch_bounds__(256) void combine_backward_kernel(const void* __restrict__ dY, const void* Z, int64_t rows,
                                                               int row_v, const int32_t* __restrict__ positions, int slots,
                                                               const float* __restrict__ weights, void* dZ,
                                                               float* __restrict__ dw) {
  using P = Piece<BF16, VEC>;
  __shared__ float sums[4][kSlotsAtOnce];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.x;
  for (int j0 = 0; j0 < slots; j0 += kSlotsAtOnce) {
    Slots4 s;
    s.load(positions, weights, t * slots + j0, slots - j0, rows);
    float dot[kSlotsAtOnce] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = threadIdx.x; c < row_v; c += 256) {
      P y, z[kSlotsAtOnce];
      y.load(dY, t * row_v + c);
      if (dw) {  // every load before the first store: dZ may be Z
#pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j)
          if (s.p[j] >= 0) z[j].load(Z, s.p[j] * row_v + c);
#pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j)
          if (s.p[j] >= 0) {
#pragma unroll
            for (int i = 0; i < P::kN; ++i) dot[j] = fmaf(y.v[i], z[j].v[i], dot[j]);
          }
      }
      if (dZ) {
#pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j)
          if (s.p[j] >= 0) {
            P d;
#pragma unroll
            for (int i = 0; i < P::kN; ++i) d.v[i] = s.w[j] * y.v[i];
            d.store(dZ, s.p[j] * row_v + c);
          }
      }
    }
    if (dw) {
#pragma unroll
      for (int j = 0; j < kSlotsAtOnce; ++j) {
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) dot[j] += __shfl_xor(dot[j], off);
        if (lane == 0) sums[wave][j] = dot[j];
      }
      __syncthreads();
      const int j = threadIdx.x;
      if (j < kSlotsAtOnce && j0 + j < slots)
        dw[t * slots + j0 + j] = ((sums[0][j] + sums[1][j]) + sums[2][j]) + sums[3][j];
      __syncthreads();
    }
  }
}

// Segments of a sort's first launch; 0: one launch
constexpr int64_t kOneLaunchSlots = 4096, kMostSegments = 256;
int64_t sort_segments(int64_t N) {
  return N <= kOneLaunchSlots ? 0 : ceil_div(N, 4096) < kMostSegments ? ceil_div(N, 4096) : kMostSegments;
}

// Rows as the kernels take them: n pieces of 16 bytes, or of one entry, `threads` to a workgroup
struct RowShape {
  bool vec;
  int64_t n;
  int threads;
  RowShape(int64_t D, int size) : vec(D * size % 16 == 0), n(vec ? D * size / 16 : D), threads((int)(n > 192 ? 256 : ceil_div(n, kWave) * kWave)) {}
  dim3 grid(int64_t T) const { return dim3((unsigned)T, (unsigned)ceil_div(n, threads)); }
};

}  // namespace

size_t tokens_sort_workspace_bytes(int64_t N, int64_t experts) { return (size_t)(sort_segments(N) * experts) * sizeof(int); }

bool tokens_grids_fit(int64_t T, int64_t D, int size) { return T == 0 || grid_fits(RowShape(D, size).grid(T), 256); }

hipError_t launch_tokens_sort(const void* ids, bool wide, int64_t N, int64_t experts, int32_t* offsets, int32_t* positions,
                              void* workspace, hipStream_t stream) {
  const int64_t segments = sort_segments(N);
  const int64_t segment = segments ? ceil_div(ceil_div(N, segments), 64) * 64 : N;
  const unsigned blocks = segments ? (unsigned)ceil_div(N, segment) : 1;
  int* const counts = segments ? (int*)workspace : nullptr;
  if (segments) {
    count_kernel<<<dim3(blocks), dim3(kSortThreads), experts * sizeof(int), stream>>>(ids, wide, N, segment, (int)experts, counts);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  place_kernel<<<dim3(blocks), dim3(kSortThreads), (kSortWaves + 2) * experts * sizeof(int), stream>>>(
      ids, wide, N, segment, (int)experts, counts, offsets, positions);
  return hipGetLastError();
}

hipError_t launch_tokens_gather(const void* X, int64_t T, int64_t D, int size, const int32_t* positions, int64_t slots, void* Xs,
                                int64_t rows, hipStream_t stream) {
  const RowShape r(D, size);
  const auto launch = [&](auto v) {
    using V = decltype(v);
    gather_kernel<V><<<r.grid(T), dim3(r.threads), 0, stream>>>((const V*)X, (int)r.n, positions, (int)slots, (V*)Xs, rows);
  };
  if (r.vec) launch(u32x4_t{});
  else if (size == 4) launch(uint32_t{});
  else if (size == 2) launch(uint16_t{});
  else launch(uint8_t{});
  return hipGetLastError();
}

hipError_t launch_tokens_combine(const void* Z, int64_t rows, int64_t D, bool bf16, const int32_t* positions, int64_t T,
                                 int64_t slots, const float* weights, const void* residual, void* Y, hipStream_t stream) {
  const RowShape r(D, bf16 ? 2 : 4);
  const auto kernel = bf16 ? (r.vec ? combine_kernel<true, true> : combine_kernel<true, false>)
                           : (r.vec ? combine_kernel<false, true> : combine_kernel<false, false>);
  kernel<<<r.grid(T), dim3(r.threads), 0, stream>>>(Z, rows, (int)r.n, positions, (int)slots, weights, residual, Y);
  return hipGetLastError();
}

hipError_t launch_tokens_combine_backward(const void* dY, const void* Z, int64_t rows, int64_t D, bool bf16,
                                          const int32_t* positions, int64_t T, int64_t slots, const float* weights, void* dZ,
                                          float* dweights, hipStream_t stream) {
  const RowShape r(D, bf16 ? 2 : 4);
  const auto kernel = bf16 ? (r.vec ? combine_backward_kernel<true, true> : combine_backward_kernel<true, false>)
                           : (r.vec ? combine_backward_kernel<false, true> : combine_backward_kernel<false, false>);
  kernel<<<dim3((unsigned)T), dim3(256), 0, stream>>>(dY, Z, rows, (int)r.n, positions, (int)slots, weights, dZ, dweights);
  return hipGetLastError();
}

}  // namespace splr
