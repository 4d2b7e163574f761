// Which kernels take a call of the layer product with a fused epilogue (splr_linear_fused,
// splr_linear_experts).
#include <algorithm>
#include <cmath>

#include "common.hpp"
#include "groups.hpp"
#include "kernels.hpp"

namespace splr {
namespace {

int64_t few_token_blocks(const FusedCall& c, int64_t tokens) {
  return c.offsets ? most_group_tiles(c.M, c.experts, tokens) : ceil_div(c.M, tokens);
}

// The path with the least predicted time, from whole-call times on MI355X (256 CUs) over n_in 512 ..
// 14336, n_out 1003 .. 14336, 16 .. 1024 rows and 6 .. 60 experts of 1 .. 160 rows. A workgroup costs a
// fixed part and a part per 64-column step; workgroups run 256 at a time (the small ones of the few-token
// kernels pack into any fraction of that); nothing is faster than reading S. Examples, bfloat16, us by path
// (16 tokens / 32 tokens / 128 x 64 tiles / 256 x 128 tiles):
//   4096 -> 4096    65 rows    32 /  29 /  31 /  47        256 rows     88 /  68 /  31 /  50
//   4096 -> 14336  128 rows   150 / 115 /  33 /  50        700 rows    724 / 532 / 124 / 110
//   1056 -> 1003   256 rows    22 /  19 /  27 /  39        700 rows     47 /  36 /  28 /  40
//   60 experts 2048 -> 1408, 2 rows each  57 / 73 / 53 / 64;  16 rows  92 / 86 / 58 / 67;  100 rows  391 /
//   295 / 101 / 88. float32 (three paths), 4096 -> 4096: 32 rows 37 / 31 / 74, 128 rows 106 / 86 / 76.
FusedPath path_of(const FusedCall& c) {
  const double steps = (double)ceil_div(c.n_in, 64);
  const double active = (double)std::min(c.experts, c.M);  // experts with rows, about
  // row blocks of all experts, each one's last about half full
  const auto blocks = [&](int64_t rows) {
    return c.offsets ? std::max(active, (double)c.M / rows + active / 2) : (double)ceil_div(c.M, rows);
  };
  const double read = active * c.n_out * c.n_in * (c.bf16 ? 1.125 : 2.125) / 4.5e6;  // S at 4.5 TB/s, us
  const double never = 1e30;
  const auto few_tokens = [&](int64_t tokens, double each) {
    if (few_token_blocks(c, tokens) > 65535) return never;  // a grid's second dimension
    if (few_token_pairs(c, tokens)) each *= 0.87;
    return std::max(std::max(1.0, (double)ceil_div(c.n_out, 16) / 256 * blocks(tokens)) * each, read) + 6;
  };
  const double t16 = few_tokens(16, c.bf16 ? 0.8 + 0.06 * steps : 1.0 + 0.18 * steps);
  const double t32 = few_tokens(32, c.bf16 ? 1.3 + 0.1 * steps : 2.0 + 0.28 * steps);
  const double tile_rounds = std::ceil(blocks(64) * ceil_div(c.n_out, 128) / 256);
  // a launch that the dispatch limits do not take is no choice. One path always fits: with the tiles past the
  // limits n_out is 2^20 or more, so there are few rows, and the few-token kernels take these
  const double tile = !fused_tile_grid_fits(c) ? never
                      : c.bf16 ? std::max(tile_rounds * (3 + 0.28 * steps) - 3, read) + 14
                               : std::max(tile_rounds * (3 + 0.9 * steps) - 3, read) + 18;
  const double steps4 = (double)(ceil_div(c.n_in, 256) * 4);  // the prefill kernel's loop pads to four steps
  const double wide_rounds = std::ceil(blocks(128) * ceil_div(c.n_out, 256) / 256);
  const double prefill = c.bf16 && fused_prefill_grid_fits(c) ? std::max(wide_rounds * 0.7 * steps4, read) + 14 : never;
  const double best = std::min(std::min(t16, t32), std::min(tile, prefill));
  if (t16 == best) return FusedPath::kTokens16;
  if (t32 == best) return FusedPath::kTokens32;
  return tile == best ? FusedPath::kTile : FusedPath::kPrefill;
}

}  // namespace

bool prepare_fused(FusedCall& c) {
  c.path = path_of(c);
  c.slices = c.r == 0 ? 1 : c.bf16 ? fused_lowrank_slices(c) : f32_lowrank_slices(c);
  if (c.r > 0 && !(c.bf16 ? fused_lowrank_grid_fits(c) : f32_lowrank_grid_fits(c))) return false;
  if (c.path == FusedPath::kPrefill) return fused_prefill_grid_fits(c);
  if (c.path == FusedPath::kTile) return fused_tile_grid_fits(c);
  return grid_fits(dim3((unsigned)ceil_div(c.n_out, 16)), 256);
}

size_t fused_workspace_bytes(const FusedCall& c) { return (size_t)c.slices * c.M * c.r * sizeof(float); }

FusedTile fused_tile(const FusedCall& c) {
  if (c.path == FusedPath::kPrefill) return {fused_prefill_rows(c), 128};
  if (c.path == FusedPath::kTile) return {128, 64};
  const int tokens = c.path == FusedPath::kTokens16 ? 16 : 32;
  return {few_token_pairs(c, tokens) ? 32 : 16, tokens};
}

hipError_t launch_fused(const FusedCall& c, hipStream_t stream) {
  if (c.r > 0) {
    const hipError_t e = c.bf16 ? launch_fused_lowrank(c, stream) : launch_f32_lowrank(c, stream);
    if (e != hipSuccess) return e;
  }
  if (c.path == FusedPath::kPrefill) return launch_fused_prefill(c, stream);
  if (c.path == FusedPath::kTile) return launch_fused_tile(c, stream);
  const int tokens = c.path == FusedPath::kTokens16 ? 16 : 32;
  return c.bf16 ? launch_fused_decode(c, tokens, stream) : launch_fused_decode_f32(c, tokens, stream);
}

}  // namespace splr
