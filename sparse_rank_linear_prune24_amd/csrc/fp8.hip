// Which kernels take a call of the product with 8-bit weights (splr_linear_fp8, splr_linear_fp8_experts).
#include "fp8.hpp"

namespace splr {

bool plan_fp8(const Fp8Call& c, Fp8Plan* plan) {
  *plan = Fp8Plan{false, 16, 16};
  return fp8_few_grid_fits(c);
}

size_t fp8_workspace_bytes(const Fp8Call& c, const Fp8Plan& plan) {
  return plan.quantize ? (size_t)c.M * c.n_in + (size_t)c.M * ceil_div(c.n_in, kBlockK) * sizeof(float) : 0;
}

hipError_t launch_fp8(const Fp8Call& c, const Fp8Plan& plan, hipStream_t stream) {
  (void)plan;
  return launch_fp8_few(c, stream);
}

}  // namespace splr
