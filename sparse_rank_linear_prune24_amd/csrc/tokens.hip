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
// Rows are copied by the sort's launch where one workgroup sorts and there is as little to copy: its 16 waves take a row at a
// time. Whole calls in a graph, 32 experts, bfloat16 rows, copied by the sort / by a launch of their own, us:
//   128 columns   8 slots 3.8 / 4.8    64 slots 4.8 / 5.3    128 slots 6.0 / 5.3    256 slots 8.3 / 5.4
//   1024 columns  8 slots 4.0 / 4.7    32 slots (64 KiB) 4.8 / 5.2    64 slots 5.7 / 5.2
//   2048 columns  8 slots 4.3 / 4.8    16 slots (64 KiB) 4.7 / 5.2    32 slots 5.7 / 5.3      7168 columns  8 slots 5.8 / 5.2
constexpr int kCopySlots = 64, kCopyBytes = 64 << 10;

// A slot's expert, -1 when its id names none.
__device__ __forceinline__ int expert_of(const void* ids, int wide, int64_t i, int experts) {
  const int64_t id = wide ? ((const int64_t*)ids)[i] : ((const int32_t*)ids)[i];
  return id >= 0 && id < experts ? (int)id : -1;
}

// The lanes of a wave that have this lane's expert, e >= 0 (all lanes call)
__device__ __forceinline__ uint64_t same_expert(int e, int bits) {
  uint64_t same = __ballot(e >= 0);
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((e >> b) & 1);
    same &= ((e >> b) & 1) ? set : ~set;
  }
  return same;
}

// counts[e] += slots first .. last-1 with id e, by `threads` threads (integer sums: their order does not matter). One addition a
// slot: adding once for each expert of a wave instead, found with a ballot for each bit of the ids, measured slower for 8
// experts as well (16384 slots in one launch 16 instead of 10 us).
__device__ __forceinline__ void count_slots(const void* ids, int wide, int64_t first, int64_t last, int experts, int* counts,
                                            int tid, int threads) {
  constexpr int kAtOnce = 4;
  for (int64_t i0 = first + tid; i0 < last; i0 += (int64_t)threads * kAtOnce) {
    int e[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int64_t i = i0 + (int64_t)u * threads;
      e[u] = i < last ? expert_of(ids, wide, i, experts) : -1;
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u)
      if (e[u] >= 0) atomicAdd(counts + e[u], 1);
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

// Exclusive prefix sum over the workgroup's threads, thread after thread. sums: one for each wave
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

// Turns the waves' counts [waves][experts] of each expert into where their first slots go, from `at` on; returns their sum.
__device__ __forceinline__ int places_of_waves(int* next, int waves, int experts, int e, int at) {
  int c[kSortWaves], sum = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) c[w] = w < waves ? next[w * experts + e] : 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    if (w < waves) next[w * experts + e] = at + sum;
    sum += c[w];
  }
  return sum;
}

// Positions of one segment of slots a workgroup, and the offsets. counts: every segment's counts; NULL: each workgroup counts
// all N slots itself, which saves the first launch where N is small.
__global__ __launch_bounds__(kSortThreads) void place_kernel(const void* __restrict__ ids, int wide, int64_t N, int64_t segment,
                                                             int experts, const int* __restrict__ counts,
                                                             int32_t* __restrict__ offsets, int32_t* __restrict__ positions) {
  extern __shared__ int lds[];
  __shared__ int sums[kSortWaves];
  int* const next = lds;                           // [waves][experts]: where a wave's next slot of an expert goes
  int* const before = lds + kSortWaves * experts;  // slots of the segments before
  int* const others = before + experts;            // and of those behind
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
      int b = 0, o = 0;
      for (int s = 0; s < segments; ++s) {
        const int c = counts[(size_t)s * experts + e];
        b += s < (int)blockIdx.x ? c : 0;
        o += s > (int)blockIdx.x ? c : 0;
      }
      before[e] = b;
      others[e] = o;
    }
  } else {
    count_slots(ids, wide, 0, first, experts, before, tid, kSortThreads);
    count_slots(ids, wide, last, N, experts, others, tid, kSortThreads);
  }
  __syncthreads();
  int total = 0;
  if (tid < experts) total = before[tid] + places_of_waves(next, kSortWaves, experts, tid, 0) + others[tid];
  const int start = prefix_of_block(total, sums);
  if (tid < experts) {
    if (blockIdx.x == 0) {
      offsets[tid] = start;
      if (tid == experts - 1) offsets[experts] = start + total;
    }
    before[tid] += start;
  }
  __syncthreads();
  const int bits = 32 - __builtin_clz(experts | 1);
  int* const mine_next = next + wave * experts;
  for (int64_t i0 = w_first; i0 < w_last; i0 += kWave) {
    const int64_t i = i0 + lane;
    const int e = i < w_last ? expert_of(ids, wide, i, experts) : -1;
    const uint64_t same = same_expert(e, bits);
    int at = -1;
    const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
    if (e >= 0) at = mine_next[e] + rank;
    // every lane has read before one of each expert writes, and that before the next round's reads
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (e >= 0 && rank == 0) mine_next[e] = at + __popcll(same);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (i < w_last) positions[i] = e >= 0 ? before[e] + at : -1;
  }
}

// The whole sort of at most 1024 slots by one workgroup, a slot a thread, for decoding: ids are read once. X: rows of row_v pieces
// to copy to Xs besides (NULL: by another launch).
__global__ __launch_bounds__(kSortThreads) void place_few_kernel(const void* __restrict__ ids, int wide, int N, int experts,
                                                                 int32_t* __restrict__ offsets, int32_t* __restrict__ positions,
                                                                 const u32x4_t* __restrict__ X, u32x4_t* __restrict__ Xs,
                                                                 int row_v, int slots) {
  extern __shared__ int lds[];  // [waves][experts], then where each expert starts
  __shared__ int sums[kSortWaves], placed[kCopySlots];
  const int tid = threadIdx.x, threads = blockDim.x, waves = threads / kWave, lane = tid & 63, wave = tid >> 6;
  const int e = tid < N ? expert_of(ids, wide, tid, experts) : -1;
  for (int i = tid; i < waves * experts; i += threads) lds[i] = 0;
  const uint64_t same = same_expert(e, 32 - __builtin_clz(experts | 1));
  const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
  int* const starts = lds + waves * experts;
  __syncthreads();
  if (e >= 0 && rank == 0) lds[wave * experts + e] = __popcll(same);
  __syncthreads();
  const int total = tid < experts ? places_of_waves(lds, waves, experts, tid, 0) : 0;
  const int start = prefix_of_block(total, sums);
  if (tid < experts) {
    offsets[tid] = starts[tid] = start;
    if (tid == experts - 1) offsets[experts] = start + total;
  }
  __syncthreads();
  const int at = e >= 0 ? starts[e] + lds[wave * experts + e] + rank : -1;
  if (tid < N) positions[tid] = at;
  if (!X) return;
  if (tid < N) placed[tid] = at;
  __syncthreads();
  for (int j = wave; j < N; j += waves) {  // a wave a slot
    const int to = placed[j];
    if (to < 0) continue;
    const u32x4_t* const from = X + (int64_t)(j / slots) * row_v;
    for (int c = lane; c < row_v; c += kWave) Xs[(int64_t)to * row_v + c] = from[c];
  }
}

// ------------------------------------------------------------------------------------------------- rows

// Rows are taken in pieces of 16 bytes. Rows that are not a multiple of that start anywhere (at an entry's alignment, which
// the loads and stores of gfx950 take), and their last piece, with `left` entries, is taken one by one.
__device__ __forceinline__ u32x4_t load16(const void* p) {
  u32x4_t v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

template <typename T>  // an entry, of 1, 2 or 4 bytes
__global__ __launch_bounds__(256) void gather_kernel(const T* __restrict__ X, int D, const int32_t* __restrict__ positions,
                                                     int slots, T* __restrict__ Xs, int64_t rows) {
  constexpr int kN = 16 / sizeof(T);
  const int64_t t = blockIdx.x;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * kN, left = D - c;
  if (left <= 0) return;
  const T* const from = X + t * D + c;
  u32x4_t v;
  T one[kN];
  if (left >= kN) {
    v = load16(from);
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) one[i] = i < left ? from[i] : T(0);
  }
  for (int j = 0; j < slots; ++j) {
    const int64_t p = positions[t * slots + j];
    if (p < 0 || p >= rows) continue;
    T* const to = Xs + p * D + c;
    if (left >= kN) {
      __builtin_memcpy(to, &v, 16);
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (i < left) to[i] = one[i];
    }
  }
}

// Eight bfloat16 or four float32 entries from entry `at` on, of which `left` exist (the others read as 0)
template <bool BF16>
struct Piece {
  static constexpr int kN = BF16 ? 8 : 4;
  float v[kN];
  __device__ __forceinline__ void load(const void* p, int64_t at, int left) {
    if (left >= kN) {
      const u32x4_t w = load16(BF16 ? (const void*)((const uint16_t*)p + at) : (const void*)((const float*)p + at));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (BF16) {
          v[2 * i] = __uint_as_float(w[i] << 16);
          v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        } else {
          v[i] = __uint_as_float(w[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        v[i] = 0.0f;
        if (i < left) v[i] = BF16 ? bf16_bits_to_float(((const uint16_t*)p)[at + i]) : ((const float*)p)[at + i];
      }
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t at, int left) const {
    u32x4_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BF16) w[i] = round_bf16x2(v[2 * i], v[2 * i + 1]);
      else w[i] = __float_as_uint(v[i]);
    }
    if (left >= kN) {
      __builtin_memcpy(BF16 ? (void*)((uint16_t*)p + at) : (void*)((float*)p + at), &w, 16);
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (i < left) {
          if constexpr (BF16) ((uint16_t*)p)[at + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
          else ((float*)p)[at + i] = v[i];
        }
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

template <bool BF16>
__global__ __launch_bounds__(256) void combine_kernel(const void* __restrict__ Z, int64_t rows, int D,
                                                      const int32_t* __restrict__ positions, int slots,
                                                      const float* __restrict__ weights, const void* residual, void* Y) {
  using P = Piece<BF16>;
  const int64_t t = blockIdx.x;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * P::kN, left = D - c;
  if (left <= 0) return;
  P sum, r;
#pragma unroll
  for (int i = 0; i < P::kN; ++i) sum.v[i] = 0.0f;
  if (residual) r.load(residual, t * D + c, left);
  for (int j0 = 0; j0 < slots; j0 += kSlotsAtOnce) {
    Slots4 s;
    s.load(positions, weights, t * slots + j0, slots - j0, rows);
    P z[kSlotsAtOnce];
#pragma unroll
    for (int j = 0; j < kSlotsAtOnce; ++j)
      if (s.p[j] >= 0) z[j].load(Z, s.p[j] * D + c, left);
#pragma unroll
    for (int j = 0; j < kSlotsAtOnce; ++j)
      if (s.p[j] >= 0) {
#pragma unroll
        for (int i = 0; i < P::kN; ++i) sum.v[i] = fmaf(s.w[j], z[j].v[i], sum.v[i]);
      }
  }
  if (residual) {
#pragma unroll
    for (int i = 0; i < P::kN; ++i) sum.v[i] += r.v[i];
  }
  sum.store(Y, t * D + c, left);
}

// One workgroup a token: dY's row is read once for every four slots (from L1 after the first).
template <bool BF16>
__global__ __launch_bounds__(256) void combine_backward_kernel(const void* __restrict__ dY, const void* Z, int64_t rows, int D,
                                                               const int32_t* __restrict__ positions, int slots,
                                                               const float* __restrict__ weights, void* dZ,
                                                               float* __restrict__ dw) {
  using P = Piece<BF16>;
  __shared__ float sums[4][kSlotsAtOnce];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int64_t t = blockIdx.x;
  for (int j0 = 0; j0 < slots; j0 += kSlotsAtOnce) {
    Slots4 s;
    s.load(positions, weights, t * slots + j0, slots - j0, rows);
    float dot[kSlotsAtOnce] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int c = threadIdx.x * P::kN; c < D; c += blockDim.x * P::kN) {
      const int left = D - c;
      P y, z[kSlotsAtOnce];
      y.load(dY, t * D + c, left);
      if (dw) {  // every load before the first store: dZ may be Z
#pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j)
          if (s.p[j] >= 0) z[j].load(Z, s.p[j] * D + c, left);
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
            d.store(dZ, s.p[j] * D + c, left);
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
      if (j < kSlotsAtOnce && j0 + j < slots) {
        float sum = sums[0][j];
        for (int w = 1; w < waves; ++w) sum += sums[w][j];
        dw[t * slots + j0 + j] = sum;
      }
      __syncthreads();
    }
  }
}

// How a sort of N slots is cut. Up to kOneLaunch slots every workgroup counts all of them itself; beyond, a launch of its own
// counts each segment. Whole calls in a graph, one launch / two, us:
//   8 experts     4096 slots 4.8 / 6.3    8192 5.9 / 6.9    16384 7.5 / 7.9    24576 9.2 / 8.8     32768 10.7 / 9.6    65536 17.2 / 13.1
//   64 experts    4096 slots 4.9 / 7.0    8192 5.7 / 8.3    16384 7.0 / 10.3   24576 8.4 / 12.1    32768 9.7 / 13.9    65536 15.3 / 20.1
//   1024 experts  4096 slots 6.4 / 8.9    8192 7.1 / 10.1   16384 8.5 / 12.0   24576 9.9 / 14.0    32768 11.1 / 15.9   65536 16.6 / 23.6
// The limit is where few experts, whose slots meet on few counters, stop gaining; many would gain beyond it too.
constexpr int64_t kOneLaunch = 16384, kSegment = 1024, kMostSegments = 256;
struct SortShape {
  int64_t segment;
  unsigned segments;
  bool counted;  // by a launch of its own
  explicit SortShape(int64_t N) : counted(N > kOneLaunch) {
    const int64_t wanted = ceil_div(N, kSegment), most = wanted < kMostSegments ? wanted : kMostSegments;
    segment = N == 0 ? 0 : ceil_div(ceil_div(N, most), 64) * 64;
    segments = N == 0 ? 1u : (unsigned)ceil_div(N, segment);
  }
};
dim3 row_grid(int64_t T, int64_t D, int size, unsigned* threads) {
  const int64_t pieces = ceil_div(D * size, 16);
  *threads = (unsigned)(pieces > 192 ? 256 : ceil_div(pieces, kWave) * kWave);
  return dim3((unsigned)T, (unsigned)ceil_div(pieces, *threads));
}

}  // namespace

size_t tokens_sort_workspace_bytes(int64_t N, int64_t experts) {
  const SortShape s(N);
  return s.counted ? (size_t)s.segments * experts * sizeof(int) : 0;
}

bool tokens_grids_fit(int64_t T, int64_t D, int size) {
  unsigned threads;
  return T == 0 || grid_fits(row_grid(T, D, size, &threads), 256);
}

hipError_t launch_tokens_dispatch(const void* ids, bool wide, int64_t T, int64_t slots, int64_t experts, int32_t* offsets,
                                  int32_t* positions, void* workspace, const void* X, int64_t D, int size, void* Xs,
                                  hipStream_t stream) {
  const int64_t N = T * slots;
  hipError_t e;
  bool copies = false;
  if (N <= kSortThreads) {
    copies = X && N <= kCopySlots && D * size % 16 == 0 && N * D * size <= kCopyBytes;
    // a thread each slot and each expert's prefix, a wave each row
    const int64_t most = N > experts ? N : experts, wanted = ceil_div(most, kWave) * kWave;
    const int threads = copies ? kSortThreads : (int)(wanted > 256 ? wanted : 256);
    place_few_kernel<<<dim3(1), dim3(threads), (threads / kWave + 1) * experts * sizeof(int), stream>>>(
        ids, wide, (int)N, (int)experts, offsets, positions, copies ? (const u32x4_t*)X : nullptr, (u32x4_t*)Xs,
        (int)(D * size / 16), (int)slots);
    e = hipGetLastError();
  } else {
    const SortShape s(N);
    int* const counts = s.counted ? (int*)workspace : nullptr;
    if (s.counted) {
      count_kernel<<<dim3(s.segments), dim3(kSortThreads), experts * sizeof(int), stream>>>(ids, wide, N, s.segment, (int)experts, counts);
      e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    place_kernel<<<dim3(s.segments), dim3(kSortThreads), (kSortWaves + 2) * experts * sizeof(int), stream>>>(
        ids, wide, N, s.segment, (int)experts, counts, offsets, positions);
    e = hipGetLastError();
  }
  if (e != hipSuccess || !X || copies || T == 0) return e;
  return launch_tokens_gather(X, T, D, size, positions, slots, Xs, N, stream);
}

hipError_t launch_tokens_gather(const void* X, int64_t T, int64_t D, int size, const int32_t* positions, int64_t slots, void* Xs,
                                int64_t rows, hipStream_t stream) {
  unsigned threads;
  const dim3 grid = row_grid(T, D, size, &threads);
  const auto launch = [&](auto entry) {
    using V = decltype(entry);
    gather_kernel<V><<<grid, dim3(threads), 0, stream>>>((const V*)X, (int)D, positions, (int)slots, (V*)Xs, rows);
  };
  if (size == 4) launch(uint32_t{});
  else if (size == 2) launch(uint16_t{});
  else launch(uint8_t{});
  return hipGetLastError();
}

hipError_t launch_tokens_combine(const void* Z, int64_t rows, int64_t D, bool bf16, const int32_t* positions, int64_t T,
                                 int64_t slots, const float* weights, const void* residual, void* Y, hipStream_t stream) {
  unsigned threads;
  const dim3 grid = row_grid(T, D, bf16 ? 2 : 4, &threads);
  const auto kernel = bf16 ? combine_kernel<true> : combine_kernel<false>;
  kernel<<<grid, dim3(threads), 0, stream>>>(Z, rows, (int)D, positions, (int)slots, weights, residual, Y);
  return hipGetLastError();
}

hipError_t launch_tokens_combine_backward(const void* dY, const void* Z, int64_t rows, int64_t D, bool bf16,
                                          const int32_t* positions, int64_t T, int64_t slots, const float* weights, void* dZ,
                                          float* dweights, hipStream_t stream) {
  unsigned threads;
  row_grid(T, D, bf16 ? 2 : 4, &threads);
  const auto kernel = bf16 ? combine_backward_kernel<true> : combine_backward_kernel<false>;
  kernel<<<dim3((unsigned)T), dim3(threads), 0, stream>>>(dY, Z, rows, (int)D, positions, (int)slots, weights, dZ, dweights);
  return hipGetLastError();
}

}  // namespace splr
