// Which kernels take a call of the product with 8-bit weights (splr_linear_fp8, splr_linear_fp8_experts).
#include "fp8.hpp"

namespace splr {

bool plan_fp8(const Fp8Call& c, Fp8Plan* plan) {
  const int64_t rows_each = c.offsets ? ceil_div(c.M, c.experts) : c.M;
  if (rows_each <= 32) {
    *plan = Fp8Plan{false, 16, 16};
    return fp8_few_grid_fits(c);
  }
  const int64_t big = c.y_bf16 ? 256 : 128;
  if (ceil_div(c.n_out, 256) * (ceil_div(c.M, big) + (c.offsets ? c.experts / 2 : 0)) >= 192) *plan = Fp8Plan{c.x_type != 2, 256, (int)big};
  else *plan = Fp8Plan{c.x_type != 2, 128, 128};
  return fp8_tile_grid_fits(c, plan->rows, plan->tokens) &&
         (!plan->quantize || fp8_quantize_grids_fit(c.M, c.n_in, false, false));
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
  return plan.rows > 32 ? launch_fp8_tile(q, plan.rows, stream) : launch_fp8_few(q, stream);
}

}  // namespace splr
