// Which kernels take a call of the product with 8-bit weights (splr_linear_fp8, splr_linear_fp8_experts).
#include <algorithm>
#include <cmath>

#include "fp8.hpp"

namespace splr {

// The path with the least predicted time, from whole-call times on MI355X (256 CUs) over n_in 1056 .. 14336, n_out 1003 ..
// 14336, 16 .. 4096 rows, and 4 .. 60 experts of 2 .. 380 rows, X in bfloat16. A step is a block of 128 columns. Examples, us by
// path (few-token kernel with 16 / 32 tokens a workgroup; tiles of 128 x 128 with two / four steps in LDS; of 256 x 256):
//   4096 -> 4096, bfloat16 Y     16 rows  10 /  11 / 30 / 26 / 49     128 rows  29 / 21 / 32 / 27 / 50
//                               512 rows  95 /  63 / 34 / 29 / 53    4096 rows    -  / - / 96 / 119 / 79
//   4096 -> 14336               256 rows 152 /  97 / 34 / 30 / 50    2048 rows    -  / - / 178 / 190 / 134
//   14336 -> 1024               256 rows  42 /  31 / 94 / 73 / 149
//   96 -> 13120                 224 rows  92 with 16 tokens a workgroup
//   8 experts 4096 -> 4096, 8 rows each 46 / 46 / 51 / 44 / 59; 300 rows each 726 / 473 / 98 / 91 / 75
// float32 Y (no tiles of 256): 4096 -> 4096, 512 rows 94 / 62 / 42 / 41, 4096 rows -/-/ 150 / 176.
bool plan_fp8(const Fp8Call& c, Fp8Plan* plan) {
  const double KB = (double)ceil_div(c.n_in, kBlockK), active = (double)std::min(c.experts, c.M);
  // row blocks of all experts, each one's last about half full
  const auto blocks = [&](int tokens) {
    return c.offsets ? std::max(active, (double)c.M / tokens + active / 2) : (double)ceil_div(c.M, tokens);
  };
  const double read = active * c.n_out * c.n_in / 4.0e6 + 8;  // W at 4 TB/s, us
  const double never = 1e30;
  // a workgroup's part of a tile of 16 rows: its meeting and store, and the blocks of its tokens
  const auto few = [&](int tokens, double fixed, double tile, double block) {
    if (!fp8_few_grid_fits(c, tokens)) return never;
    return std::max(fixed + blocks(tokens) * ceil_div(c.n_out, 16) * (tile + block * KB), read);
  };
  const double t16 = few(16, 6.5, 5.5e-3, 0.24e-3), t32 = few(32, 8.6, 5e-3, 0.33e-3);
  // one workgroup a CU: four steps in LDS hide its latencies; more: two steps, so that a CU takes two
  const double tiles = blocks(128) * ceil_div(c.n_out, 128);
  const int stages = tiles <= 256 ? 4 : 2;
  const double step = c.y_bf16 ? (stages == 4 ? 0.55 : 1.4) : (stages == 4 ? 0.85 : 2.0);
  const double t128 =
      !fp8_tile_grid_fits(c, 128, 128) ? never : std::max(8 + std::ceil(stages == 4 ? 1 : tiles / 512) * (3 + step * KB), read);
  const double wide = blocks(256) * ceil_div(c.n_out, 256);
  const double t256 = !c.y_bf16 || c.w_rows || !fp8_tile_grid_fits(c, 256, 256)
                          ? never
                          : std::max(8 + std::ceil(wide / 256) * (3 + (1.25 + 0.75 * std::min(1.0, wide / 256)) * KB), read);
  const double best = std::min(std::min(t16, t32), std::min(t128, t256));
  if (best == never) return false;
  const bool quantized = c.x_type == 2;
  if (best == t16 || best == t32) {
    const int tokens = best == t16 ? 16 : 32;
    // Quantising X in every workgroup costs as much as a launch of its own (1 us) where a tile has about 112 blocks of it
    // (4096 -> 4096, one row: 7.3 instead of 8.9 us, four rows 9.5 instead of 9.0)
    const bool inside = ceil_div(c.M, c.offsets ? c.experts : 1) * KB <= 112 && fp8_few_quantizes(c, tokens);
    *plan = Fp8Plan{!quantized && !inside, 16, tokens};
  } else {
    *plan = best == t128 ? Fp8Plan{!quantized, 128, 128, stages} : Fp8Plan{!quantized, 256, 256};
  }
  return !plan->quantize || fp8_quantize_grids_fit(c.M, c.n_in, false, false);
}

size_t fp8_workspace_bytes(const Fp8Call& c, const Fp8Plan& plan) {
  return plan.quantize ? (size_t)c.M * c.n_in + (size_t)c.M * ceil_div(c.n_in, kBlockK) * sizeof(float) : 0;
}

hipError_t launch_fp8(const Fp8Call& c, const Fp8Plan& plan, hipStream_t stream) {
  Fp8Call q = c;
  if (plan.quantize) {
    float* const scales = (float*)((uint8_t*)c.workspace + c.M * c.n_in);
    const hipError_t e = launch_fp8_quantize(c.X, c.M, c.n_in, c.x_type == 1, false, false, c.workspace, scales, stream);
    if (e != hipSuccess) return e;
    q.X = c.workspace;
    q.x_scales = scales;
    q.x_type = 2;
  }
  return plan.rows == 16 ? launch_fp8_few(q, plan.tokens, stream) : launch_fp8_tile(q, plan.rows, plan.stages, stream);
}

}  // namespace splr
