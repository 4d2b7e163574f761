// Launchers of the tokens' way to their experts and back (argument checking happens in api.hip before these are called):
// N = T slots sorted by expert (ids of 4 or 8 bytes), rows of D entries of `size` bytes copied to their places, weighted and
// added back, and the gradient of that.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace splr {

size_t tokens_sort_workspace_bytes(int64_t N, int64_t experts);
bool tokens_grids_fit(int64_t T, int64_t D, int size);
// X NULL: no rows
hipError_t launch_tokens_dispatch(const void* ids, bool wide, int64_t T, int64_t slots, int64_t experts, int32_t* offsets,
                                  int32_t* positions, void* workspace, const void* X, int64_t D, int size, void* Xs,
                                  hipStream_t stream);
hipError_t launch_tokens_gather(const void* X, int64_t T, int64_t D, int size, const int32_t* positions, int64_t slots, void* Xs,
                                int64_t rows, hipStream_t stream);
hipError_t launch_tokens_combine(const void* Z, int64_t rows, int64_t D, bool bf16, const int32_t* positions, int64_t T,
                                 int64_t slots, const float* weights, const void* residual, void* Y, hipStream_t stream);
hipError_t launch_tokens_combine_backward(const void* dY, const void* Z, int64_t rows, int64_t D, bool bf16,
                                          const int32_t* positions, int64_t T, int64_t slots, const float* weights, void* dZ,
                                          float* dweights, hipStream_t stream);

}  // namespace splr
