// Which kernels take a call of the layer product with a fused epilogue (splr_linear_fused,
// splr_linear_experts).
#include <algorithm>

#include "common.hpp"
#include "groups.hpp"
#include "kernels.hpp"

namespace splr {
namespace {

// Stage 2's kernel: few tokens (decode.hip, fused_f32.hip), tiles of 128 x 64 (fused_tile.hip), or, in
// bfloat16, tiles of 256 or 512 x 128 (linear_bf16.hip).
enum class Path { kTokens16, kTokens32, kTile, kPrefill };

Path path_of(const FusedCall& c) {
  if (!c.offsets) {
    if (c.M <= 16) return Path::kTokens16;
    if (c.M <= 64) return Path::kTokens32;
    return c.bf16 ? Path::kPrefill : Path::kTile;
  }
  const int64_t mean = ceil_div(c.M, c.experts);
  if (mean <= 12) return Path::kTokens16;
  if (mean <= 24) return Path::kTokens32;
  return c.bf16 ? Path::kPrefill : Path::kTile;
}

int slices_of(const FusedCall& c) {
  if (c.r == 0) return 1;
  if (!c.bf16) return f32_lowrank_slices(c);
  return c.offsets ? experts_lowrank_slices(c) : lowrank_slices(c.M, c.n_in, c.r, true);
}

bool stage1_fits(const FusedCall& c) {
  if (c.r == 0) return true;
  if (!c.bf16) return f32_lowrank_grid_fits(c);
  return c.offsets ? experts_lowrank_grid_fits(c) : lowrank_grids_fit(c.M, c.n_in, c.r, true);
}

}  // namespace

size_t fused_workspace_bytes(const FusedCall& c) {
  return c.M == 0 || c.r == 0 ? 0 : (size_t)slices_of(c) * c.M * c.r * sizeof(float);
}

bool fused_grids_fit(const FusedCall& c) {
  if (!stage1_fits(c)) return false;
  const Path path = path_of(c);
  if (path == Path::kPrefill) return fused_prefill_grid_fits(c);
  if (path == Path::kTile) return fused_tile_grid_fits(c);
  const int64_t tokens = path == Path::kTokens16 ? 16 : 32;
  return (c.offsets ? most_group_tiles(c.M, c.experts, tokens) : ceil_div(c.M, tokens)) <= 65535 &&
         grid_fits(dim3((unsigned)ceil_div(c.n_out, 16)), 256);
}

hipError_t launch_fused(FusedCall c, hipStream_t stream) {
  c.slices = slices_of(c);
  if (c.r > 0) {
    const hipError_t e = !c.bf16    ? launch_f32_lowrank(c, stream)
                         : c.offsets ? launch_experts_lowrank(c, stream)
                                     : launch_lowrank(c.X, c.V, c.M, c.n_in, c.r, true, c.workspace, stream);
    if (e != hipSuccess) return e;
  }
  const Path path = path_of(c);
  if (path == Path::kPrefill) return launch_fused_prefill(c, stream);
  if (path == Path::kTile) return launch_fused_tile(c, stream);
  const int tokens = path == Path::kTokens16 ? 16 : 32;
  return c.bf16 ? launch_fused_decode(c, tokens, stream) : launch_fused_decode_f32(c, tokens, stream);
}

}  // namespace splr
