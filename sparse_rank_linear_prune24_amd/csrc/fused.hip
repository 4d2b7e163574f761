// Which kernels take a call of the layer product with a fused epilogue (splr_linear_fused,
// splr_linear_experts): in bfloat16 those of the plain product with the epilogue in their last step
// (lowrank.hip, decode.hip, linear_bf16.hip), in float32 those of fused_f32.hip.
#include "common.hpp"
#include "groups.hpp"
#include "kernels.hpp"

namespace splr {
namespace {

// Tokens that the decode kernel takes together, 0 where the prefill kernel is faster; for experts by the
// rows an expert has on average.
int decode_tokens(const FusedCall& c) {
  if (!c.offsets) return c.M <= kDecodeMaxTokens ? (int)c.M : 0;
  const int64_t mean = ceil_div(c.M, c.experts);
  if (mean <= 12) return 16;
  if (mean <= 24) return 32;
  return mean <= 64 ? 64 : 0;
}

int slices_of(const FusedCall& c) {
  if (c.r == 0) return 1;
  if (!c.bf16) return fused_f32_slices(c);
  return c.offsets ? experts_lowrank_slices(c) : lowrank_slices(c.M, c.n_in, c.r, true);
}

}  // namespace

size_t fused_workspace_bytes(const FusedCall& c) {
  return c.M == 0 || c.r == 0 ? 0 : (size_t)slices_of(c) * c.M * c.r * sizeof(float);
}

bool fused_grids_fit(const FusedCall& c) {
  const int tokens = decode_tokens(c);
  if (!c.bf16) return fused_f32_grids_fit(c, tokens);
  if (c.r > 0 && !(c.offsets ? experts_lowrank_grid_fits(c) : lowrank_grids_fit(c.M, c.n_in, c.r, true))) return false;
  if (!tokens) return fused_prefill_grid_fits(c);
  const int64_t block = tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64;
  return (c.offsets ? most_group_tiles(c.M, c.experts, block) : ceil_div(c.M, block)) <= 65535 &&
         grid_fits(dim3((unsigned)ceil_div(c.n_out, 16)), 256);
}

hipError_t launch_fused(FusedCall c, hipStream_t stream) {
  c.slices = slices_of(c);
  const int tokens = decode_tokens(c);
  if (!c.bf16) return launch_fused_f32(c, tokens, stream);
  if (c.r > 0) {
    const hipError_t e = c.offsets ? launch_experts_lowrank(c, stream)
                                   : launch_lowrank(c.X, c.V, c.M, c.n_in, c.r, true, c.workspace, stream);
    if (e != hipSuccess) return e;
  }
  return tokens ? launch_fused_decode(c, tokens, stream) : launch_fused_prefill(c, stream);
}

}  // namespace splr
