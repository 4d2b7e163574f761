// C ABI of libsplr (declared in include/splr.h): argument validation, workspace sizing and
// kernel dispatch.  Every check runs before the first HIP call, so a rejected call enqueues
// nothing; the library holds no mutable state and never allocates device memory.
#include "splr.h"

#include <mutex>

#include "common.hpp"
#include "fp8.hpp"
#include "kernels.hpp"
#include "tokens.hpp"

namespace {

// Size limits keep every index the kernels form inside their integer types.
constexpr int64_t kMaxRows = int64_t(1) << 24;      // n_out and M
constexpr int64_t kMaxCols = int64_t(1) << 20;      // n_in
constexpr int64_t kMaxElems = int64_t(1) << 36;     // n_out * n_in, M * n_in, M * n_out
constexpr int64_t kMaxRank = 1024;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool dtype_ok(splr_dtype_t d) { return d == SPLR_FP32 || d == SPLR_BF16; }

splr_status_t check_in(int64_t n_in) {
  return (n_in >= 32 && n_in <= kMaxCols && n_in % 32 == 0) ? SPLR_OK : SPLR_ERR_SHAPE;
}

splr_status_t check_rows(int64_t rows, int64_t n_in) {
  if (rows < 1 || rows > kMaxRows) return SPLR_ERR_SHAPE;
  if (rows * n_in > kMaxElems) return SPLR_ERR_SHAPE;
  return SPLR_OK;
}

splr_status_t check_rank(int64_t r) {
  return (r >= 0 && r <= kMaxRank && r % 16 == 0) ? SPLR_OK : SPLR_ERR_SHAPE;
}

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

size_t workspace_bytes(int64_t M, int64_t n_in, int64_t r, splr_dtype_t dtype) {
  if (r == 0) return 0;
  return round_up(splr::lowrank_workspace_bytes(M, n_in, r, dtype == SPLR_BF16), 256);
}

splr_status_t from_hip(hipError_t e) { return e == hipSuccess ? SPLR_OK : SPLR_ERR_HIP; }

}  // namespace

extern "C" {

splr_status_t splr_prune24_pack(const void* R, int64_t n_out, int64_t n_in, splr_dtype_t dtype, void* values,
                                uint32_t* meta, hipStream_t stream) {
  if (!R || !values || !meta) return SPLR_ERR_NULL;
  splr_status_t s = check_in(n_in);
  if (s == SPLR_OK) s = check_rows(n_out, n_in);
  if (s != SPLR_OK) return s;
  if (!dtype_ok(dtype)) return SPLR_ERR_DTYPE;
  if (!splr::pack_grids_fit(n_out, n_in, dtype == SPLR_BF16)) return SPLR_ERR_SHAPE;
  if (!aligned16(R) || !aligned16(values) || !aligned16(meta)) return SPLR_ERR_ALIGN;
  return from_hip(splr::launch_prune24_pack(R, n_out, n_in, dtype == SPLR_BF16, values, meta, stream));
}

splr_status_t splr_prune_nm_pack(const void* R, int64_t n_out, int64_t n_in, int32_t n, int32_t m,
                                 splr_dtype_t dtype, void* values, uint32_t* meta, hipStream_t stream) {
  if (!R || !values || !meta) return SPLR_ERR_NULL;
  splr_status_t s = check_in(n_in);
  if (s == SPLR_OK) s = check_rows(n_out, n_in);
  if (s == SPLR_OK && !((n == 1 || n == 2) && (m == 4 || m == 8 || m == 16))) s = SPLR_ERR_SHAPE;
  if (s != SPLR_OK) return s;  // n_in % 32 == 0, so every m above divides n_in
  if (!dtype_ok(dtype)) return SPLR_ERR_DTYPE;
  if (!splr::pack_grids_fit(n_out, n_in, dtype == SPLR_BF16)) return SPLR_ERR_SHAPE;
  if (!aligned16(R) || !aligned16(values) || !aligned16(meta)) return SPLR_ERR_ALIGN;
  return from_hip(splr::launch_prune_nm_pack(R, n_out, n_in, n, m, dtype == SPLR_BF16, values, meta, stream));
}

splr_status_t splr_prune24_pack_residual(const void* W, const void* U, const void* V, int64_t n_out, int64_t n_in,
                                         int64_t r, splr_dtype_t dtype, void* values, uint32_t* meta,
                                         hipStream_t stream) {
  if (!W || !values || !meta) return SPLR_ERR_NULL;
  if (r > 0 && (!U || !V)) return SPLR_ERR_NULL;
  splr_status_t s = check_in(n_in);
  if (s == SPLR_OK) s = check_rows(n_out, n_in);
  if (s == SPLR_OK && (r < 0 || r > kMaxRank)) s = SPLR_ERR_SHAPE;
  if (s != SPLR_OK) return s;
  if (!dtype_ok(dtype)) return SPLR_ERR_DTYPE;
  if (!splr::residual_grids_fit(n_out, n_in)) return SPLR_ERR_SHAPE;
  if (!aligned16(W) || !aligned16(values) || !aligned16(meta)) return SPLR_ERR_ALIGN;
  if (r > 0 && (!aligned16(U) || !aligned16(V))) return SPLR_ERR_ALIGN;
  return from_hip(
      splr::launch_prune24_pack_residual(W, U, V, n_out, n_in, r, dtype == SPLR_BF16, values, meta, stream));
}

splr_status_t splr_prune24_pack_scaled(const void* R, const float* d, int64_t n_out, int64_t n_in, splr_dtype_t dtype,
                                       void* values, uint32_t* meta, hipStream_t stream) {
  if (!R || !d || !values || !meta) return SPLR_ERR_NULL;
  splr_status_t s = check_in(n_in);
  if (s == SPLR_OK) s = check_rows(n_out, n_in);
  if (s != SPLR_OK) return s;
  if (!dtype_ok(dtype)) return SPLR_ERR_DTYPE;
  if (!splr::pack_grids_fit(n_out, n_in, dtype == SPLR_BF16)) return SPLR_ERR_SHAPE;
  if (!aligned16(R) || !aligned16(d) || !aligned16(values) || !aligned16(meta)) return SPLR_ERR_ALIGN;
  return from_hip(
      splr::launch_prune24_pack_scaled(R, d, n_out, n_in, dtype == SPLR_BF16, values, meta, stream));
}

splr_status_t splr_packed_bytes(int64_t n_out, int64_t n_in, splr_dtype_t dtype, size_t* values_bytes,
                                size_t* meta_bytes) {
  if (!values_bytes || !meta_bytes) return SPLR_ERR_NULL;
  splr_status_t s = check_in(n_in);
  if (s == SPLR_OK) s = check_rows(n_out, n_in);
  if (s != SPLR_OK) return s;
  if (!dtype_ok(dtype)) return SPLR_ERR_DTYPE;
  const size_t TR = (size_t)((n_out + 15) / 16), TK = (size_t)((n_in + 63) / 64);
  *values_bytes = TR * TK * 512 * (dtype == SPLR_BF16 ? 2 : 4);
  *meta_bytes = TR * (size_t)splr::meta_blocks((int)TK) * 1024;
  return SPLR_OK;
}

size_t splr_linear_workspace_bytes(int64_t M, int64_t n_out, int64_t n_in, int64_t r, splr_dtype_t dtype) {
  (void)n_out;
  if (M < 1 || check_in(n_in) != SPLR_OK || check_rank(r) != SPLR_OK || !dtype_ok(dtype)) return 0;
  return workspace_bytes(M, n_in, r, dtype);
}

namespace {

// Argument checks shared by splr_linear and its two stages. V is checked only when need_v, the
// caller's workspace only when check_ws.
splr_status_t check_linear(const void* X, int64_t M, int64_t n_in, const void* values, const uint32_t* meta,
                           int64_t n_out, const void* U, const void* V, int64_t r, splr_dtype_t dtype, const void* Y,
                           const void* workspace, size_t ws_bytes, bool need_sparse, bool need_v,
                           bool check_ws = true) {
  if (!X) return SPLR_ERR_NULL;
  if (need_sparse && (!values || !meta || !Y || (r > 0 && !U))) return SPLR_ERR_NULL;
  if (need_v && r > 0 && !V) return SPLR_ERR_NULL;
  splr_status_t s = check_in(n_in);
  if (s == SPLR_OK) s = check_rows(M, n_in);
  if (s == SPLR_OK && need_sparse) s = check_rows(n_out, n_in);
  if (s == SPLR_OK) s = check_rank(r);
  if (s == SPLR_OK && need_sparse && M * n_out > kMaxElems) s = SPLR_ERR_SHAPE;
  if (s != SPLR_OK) return s;
  if (!dtype_ok(dtype)) return SPLR_ERR_DTYPE;
  // every launch of the call fits the dispatch limits (stage 2 only when it runs)
  if (need_sparse ? !splr::linear_grids_fit(M, n_in, n_out, r, dtype == SPLR_BF16)
                  : !splr::lowrank_grids_fit(M, n_in, r, dtype == SPLR_BF16))
    return SPLR_ERR_SHAPE;
  if (!aligned16(X)) return SPLR_ERR_ALIGN;
  if (need_sparse && (!aligned16(values) || !aligned16(meta) || !aligned16(Y) || (r > 0 && !aligned16(U))))
    return SPLR_ERR_ALIGN;
  if (need_v && r > 0 && !aligned16(V)) return SPLR_ERR_ALIGN;
  if (!check_ws) return SPLR_OK;
  const size_t need = workspace_bytes(M, n_in, r, dtype);
  if (need > 0 && (!workspace || ws_bytes < need)) return SPLR_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return SPLR_ERR_ALIGN;
  return SPLR_OK;
}

splr_status_t run_stage2(const void* X, int64_t M, int64_t n_in, const void* values, const uint32_t* meta,
                         int64_t n_out, const void* U, int64_t r, splr_dtype_t dtype, void* Y, bool y_bf16,
                         void* workspace, hipStream_t stream) {
  if (dtype == SPLR_BF16 && M <= splr::kDecodeMaxTokens)
    return from_hip(splr::launch_linear_decode(X, M, n_in, values, meta, n_out, U, r, (const float*)workspace,
                                               splr::lowrank_slices(M, n_in, r, true), Y, y_bf16, stream));
  if (dtype == SPLR_BF16)
    return from_hip(splr::launch_linear_bf16(X, M, n_in, values, meta, n_out, U, r, (const float*)workspace,
                                             splr::lowrank_slices(M, n_in, r, true), Y, y_bf16, stream));
  return from_hip(splr::launch_linear_f32((const float*)X, M, n_in, (const float*)values, meta, n_out,
                                          (const float*)U, r, (const float*)workspace, Y, y_bf16, stream));
}

// Layers of one shape: every layer is checked as splr_linear (or its stage 2) checks it before the
// first HIP call; with stage 1 (with_stage1) each layer's T goes to its own workspace, then the
// stage-2 products run as one launch when the prefill kernel takes them, else layer by layer.
splr_status_t run_group(int32_t count, const void* const* X, int64_t M, int64_t n_in, const void* const* values,
                        const uint32_t* const* meta, int64_t n_out, const void* const* U, const void* const* V,
                        int64_t r, splr_dtype_t dtype, float* const* Y, const void* const* workspace,
                        size_t ws_bytes, bool with_stage1, hipStream_t stream) {
  static_assert(SPLR_GROUP_MAX == splr::kMaxGroup, "header and library agree");
  if (count < 1 || count > splr::kMaxGroup) return SPLR_ERR_SHAPE;
  if (!X || !values || !meta || !Y || !workspace || (r > 0 && !U) || (with_stage1 && r > 0 && !V))
    return SPLR_ERR_NULL;
  for (int32_t i = 0; i < count; ++i) {
    const splr_status_t s =
        check_linear(X[i], M, n_in, values[i], meta[i], n_out, r > 0 ? U[i] : nullptr,
                     with_stage1 && r > 0 ? V[i] : nullptr, r, dtype, Y[i], workspace[i], ws_bytes, true, with_stage1);
    if (s != SPLR_OK) return s;
  }
  const bool grouped = dtype == SPLR_BF16 && M > splr::kDecodeMaxTokens;
  if (grouped && !splr::linear_group_grid_fits(M, n_out, count)) return SPLR_ERR_SHAPE;
  if (with_stage1)
    for (int32_t i = 0; i < count; ++i)
      if (splr::launch_lowrank(X[i], V ? V[i] : nullptr, M, n_in, r, dtype == SPLR_BF16, const_cast<void*>(workspace[i]),
                               stream) != hipSuccess)
        return SPLR_ERR_HIP;
  if (!grouped) {
    for (int32_t i = 0; i < count; ++i) {
      const splr_status_t s = run_stage2(X[i], M, n_in, values[i], meta[i], n_out, r > 0 ? U[i] : nullptr, r, dtype,
                                         Y[i], false, const_cast<void*>(workspace[i]), stream);
      if (s != SPLR_OK) return s;
    }
    return SPLR_OK;
  }
  const void* u[splr::kMaxGroup];
  const float* t[splr::kMaxGroup];
  void* y[splr::kMaxGroup];
  for (int32_t i = 0; i < count; ++i) {
    u[i] = r > 0 ? U[i] : nullptr;
    t[i] = (const float*)workspace[i];
    y[i] = Y[i];
  }
  return from_hip(splr::launch_linear_bf16_group(count, X, M, n_in, values, meta, n_out, u, r, t,
                                                 splr::lowrank_slices(M, n_in, r, true), y, false, stream));
}

}  // namespace

splr_status_t splr_linear(const void* X, int64_t M, int64_t n_in, const void* values, const uint32_t* meta,
                          int64_t n_out, const void* U, const void* V, int64_t r, splr_dtype_t dtype, float* Y,
                          void* workspace, size_t ws_bytes, hipStream_t stream) {
  const splr_status_t s =
      check_linear(X, M, n_in, values, meta, n_out, U, V, r, dtype, Y, workspace, ws_bytes, true, true);
  if (s != SPLR_OK) return s;
  if (splr::launch_lowrank(X, V, M, n_in, r, dtype == SPLR_BF16, workspace, stream) != hipSuccess)
    return SPLR_ERR_HIP;
  return run_stage2(X, M, n_in, values, meta, n_out, U, r, dtype, Y, false, workspace, stream);
}

splr_status_t splr_linear_ex(const void* X, int64_t M, int64_t n_in, const void* values, const uint32_t* meta,
                             int64_t n_out, const void* U, const void* V, int64_t r, splr_dtype_t dtype,
                             splr_dtype_t y_dtype, void* Y, void* workspace, size_t ws_bytes, hipStream_t stream) {
  const splr_status_t s =
      check_linear(X, M, n_in, values, meta, n_out, U, V, r, dtype, Y, workspace, ws_bytes, true, true);
  if (s != SPLR_OK) return s;
  if (!dtype_ok(y_dtype)) return SPLR_ERR_DTYPE;
  if (splr::launch_lowrank(X, V, M, n_in, r, dtype == SPLR_BF16, workspace, stream) != hipSuccess)
    return SPLR_ERR_HIP;
  return run_stage2(X, M, n_in, values, meta, n_out, U, r, dtype, Y, y_dtype == SPLR_BF16, workspace, stream);
}

splr_status_t splr_linear_stage1(const void* X, int64_t M, int64_t n_in, const void* V, int64_t r,
                                 splr_dtype_t dtype, void* workspace, size_t ws_bytes, hipStream_t stream) {
  const splr_status_t s =
      check_linear(X, M, n_in, nullptr, nullptr, 0, nullptr, V, r, dtype, nullptr, workspace, ws_bytes, false, true);
  if (s != SPLR_OK) return s;
  return from_hip(splr::launch_lowrank(X, V, M, n_in, r, dtype == SPLR_BF16, workspace, stream));
}

splr_status_t splr_linear_stage2(const void* X, int64_t M, int64_t n_in, const void* values, const uint32_t* meta,
                                 int64_t n_out, const void* U, int64_t r, splr_dtype_t dtype, float* Y,
                                 const void* workspace, size_t ws_bytes, hipStream_t stream) {
  const splr_status_t s =
      check_linear(X, M, n_in, values, meta, n_out, U, nullptr, r, dtype, Y, workspace, ws_bytes, true, false);
  if (s != SPLR_OK) return s;
  return run_stage2(X, M, n_in, values, meta, n_out, U, r, dtype, Y, false, const_cast<void*>(workspace), stream);
}

splr_status_t splr_linear_stage2_dense(const void* X, int64_t M, int64_t n_in, const void* values,
                                       const uint32_t* meta, int64_t n_out, const void* U, int64_t r,
                                       splr_dtype_t dtype, float* Y, const void* workspace, size_t ws_bytes,
                                       hipStream_t stream) {
  const splr_status_t s =
      check_linear(X, M, n_in, values, meta, n_out, U, nullptr, r, dtype, Y, workspace, ws_bytes, true, false);
  if (s != SPLR_OK) return s;
  if (dtype != SPLR_BF16) return SPLR_ERR_DTYPE;
  if (!splr::linear_dense_grids_fit(M, n_out)) return SPLR_ERR_SHAPE;
  return from_hip(splr::launch_linear_bf16_dense(X, M, n_in, values, meta, n_out, U, r, (const float*)workspace,
                                                 splr::lowrank_slices(M, n_in, r, true), Y, stream));
}

splr_status_t splr_linear_stage2_group(int32_t count, const void* const* X, int64_t M, int64_t n_in,
                                       const void* const* values, const uint32_t* const* meta, int64_t n_out,
                                       const void* const* U, int64_t r, splr_dtype_t dtype, float* const* Y,
                                       const void* const* workspace, size_t ws_bytes, hipStream_t stream) {
  return run_group(count, X, M, n_in, values, meta, n_out, U, nullptr, r, dtype, Y, workspace, ws_bytes, false,
                   stream);
}

splr_status_t splr_linear_group(int32_t count, const void* const* X, int64_t M, int64_t n_in,
                                const void* const* values, const uint32_t* const* meta, int64_t n_out,
                                const void* const* U, const void* const* V, int64_t r, splr_dtype_t dtype,
                                float* const* Y, void* const* workspace, size_t ws_bytes, hipStream_t stream) {
  return run_group(count, X, M, n_in, values, meta, n_out, U, V, r, dtype, Y, (const void* const*)workspace,
                   ws_bytes, true, stream);
}

}  // extern "C"

// ---------------------------------------------------------------- fused epilogue, experts
namespace {

// Checks the epilogue and turns it into the kernels' form.
splr_status_t check_epilogue(const splr_epilogue_t* epilogue, splr_dtype_t dtype, splr_dtype_t y_dtype,
                             int64_t n_out, splr::Epilogue* out) {
  if (n_out > splr::kMaxFusedOut) return SPLR_ERR_SHAPE;
  if (!dtype_ok(y_dtype)) return SPLR_ERR_DTYPE;
  *out = splr::Epilogue{nullptr, nullptr, nullptr, splr::kActNone, dtype == SPLR_BF16 ? 1 : 0};
  if (!epilogue) return SPLR_OK;
  const int act = (int)epilogue->activation;
  if (act < 0 || act >= splr::kActCount) return SPLR_ERR_SHAPE;
  if (!aligned16(epilogue->bias) || !aligned16(epilogue->gate) || !aligned16(epilogue->residual))
    return SPLR_ERR_ALIGN;
  out->bias = epilogue->bias;
  out->gate = epilogue->gate;
  out->residual = epilogue->residual;
  out->act = act;
  return SPLR_OK;
}

splr::FusedCall fused_call(const void* X, int64_t M, int64_t n_in, const int32_t* offsets, int64_t experts,
                           const void* values, const uint32_t* meta, int64_t n_out, const void* U, const void* V,
                           int64_t r, splr_dtype_t dtype, const splr::Epilogue& ep, void* Y, splr_dtype_t y_dtype,
                           void* workspace) {
  return splr::FusedCall{X, M, n_in, offsets, experts, values, meta, n_out, U, V, r, dtype == SPLR_BF16, ep, Y,
                         y_dtype == SPLR_BF16, workspace};
}

// A call by its sizes, prepared, for the queries; false when it would be refused or has no rows. n_experts 0:
// splr_linear_fused.
bool query_call(int64_t M, int64_t n_experts, int64_t n_out, int64_t n_in, int64_t r, splr_dtype_t dtype,
                splr::FusedCall* c) {
  if (M < 1 || M > kMaxRows || n_out < 1 || n_out > splr::kMaxFusedOut || n_experts < 0 ||
      n_experts > SPLR_EXPERTS_MAX || check_in(n_in) != SPLR_OK || check_rank(r) != SPLR_OK || !dtype_ok(dtype))
    return false;
  const int32_t any = 0;  // a non-null `offsets`: a call by expert
  *c = fused_call(nullptr, M, n_in, n_experts ? &any : nullptr, n_experts ? n_experts : 1, nullptr, nullptr, n_out,
                  nullptr, nullptr, r, dtype, splr::Epilogue{}, nullptr, SPLR_FP32, nullptr);
  return splr::prepare_fused(*c);
}

size_t query_workspace_bytes(int64_t M, int64_t n_experts, int64_t n_out, int64_t n_in, int64_t r,
                             splr_dtype_t dtype) {
  splr::FusedCall c;
  return query_call(M, n_experts, n_out, n_in, r, dtype, &c) ? round_up(splr::fused_workspace_bytes(c), 256) : 0;
}

// Y and the workspace (`ws_bytes` of it) overlap no operand; only Y may be gate or residual itself.
splr_status_t check_overlap(const splr::FusedCall& c, size_t ws_bytes) {
  const size_t E = (size_t)c.experts, M = (size_t)c.M, n_in = (size_t)c.n_in, n_out = (size_t)c.n_out, r = (size_t)c.r;
  const size_t size = c.bf16 ? 2 : 4, y_bytes = M * n_out * (c.y_bf16 ? 2 : 4);
  const size_t TR = (n_out + 15) / 16, TK = (n_in + 63) / 64;
  struct Range {
    const void* p;
    size_t bytes;
    bool meets(const Range& o) const {
      const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
      return p && o.p && bytes && o.bytes && (a < b ? b - a < bytes : a - b < o.bytes);
    }
  };
  const Range y{c.Y, y_bytes}, workspace{c.workspace, ws_bytes};
  const Range read[] = {{c.X, M * n_in * size},
                        {c.offsets, (E + 1) * sizeof(int32_t)},
                        {c.values, E * TR * TK * 512 * size},
                        {c.meta, E * TR * (size_t)splr::meta_blocks((int)TK) * 1024},
                        {r ? c.U : nullptr, E * n_out * r * size},
                        {r ? c.V : nullptr, E * r * n_in * size},
                        {c.ep.bias, E * n_out * size}};
  for (const Range& x : read)
    if (y.meets(x) || workspace.meets(x)) return SPLR_ERR_OVERLAP;
  for (const Range& x : {Range{c.ep.gate, y_bytes}, Range{c.ep.residual, y_bytes}})
    if (workspace.meets(x) || (x.p != c.Y && y.meets(x))) return SPLR_ERR_OVERLAP;
  return workspace.meets(y) ? SPLR_ERR_OVERLAP : SPLR_OK;
}

// The last checks of a call with rows, then its launches.
splr_status_t run_fused(splr::FusedCall c, size_t ws_bytes, hipStream_t stream) {
  if (!splr::prepare_fused(c)) return SPLR_ERR_SHAPE;
  const size_t need = round_up(splr::fused_workspace_bytes(c), 256);
  if (need > 0 && (!c.workspace || ws_bytes < need)) return SPLR_ERR_WORKSPACE;
  if (need > 0 && !aligned16(c.workspace)) return SPLR_ERR_ALIGN;
  const splr_status_t s = check_overlap(c, need);
  if (s != SPLR_OK) return s;
  return from_hip(splr::launch_fused(c, stream));
}

}  // namespace

extern "C" {

size_t splr_linear_fused_workspace_bytes(int64_t M, int64_t n_out, int64_t n_in, int64_t r, splr_dtype_t dtype) {
  return query_workspace_bytes(M, 0, n_out, n_in, r, dtype);
}

splr_status_t splr_linear_fused_tile(int64_t M, int64_t n_experts, int64_t n_out, int64_t n_in, int64_t r,
                                     splr_dtype_t dtype, int32_t* rows, int32_t* tokens) {
  if (!rows || !tokens) return SPLR_ERR_NULL;
  splr::FusedCall c;
  if (!query_call(M, n_experts, n_out, n_in, r, dtype, &c)) return SPLR_ERR_SHAPE;
  const splr::FusedTile t = splr::fused_tile(c);
  *rows = t.rows;
  *tokens = t.tokens;
  return SPLR_OK;
}

splr_status_t splr_linear_fused(const void* X, int64_t M, int64_t n_in, const void* values, const uint32_t* meta,
                                int64_t n_out, const void* U, const void* V, int64_t r, splr_dtype_t dtype,
                                const splr_epilogue_t* epilogue, splr_dtype_t y_dtype, void* Y, void* workspace,
                                size_t ws_bytes, hipStream_t stream) {
  splr_status_t s =
      check_linear(X, M, n_in, values, meta, n_out, U, V, r, dtype, Y, nullptr, 0, true, true, false);
  if (s != SPLR_OK) return s;
  splr::Epilogue ep;
  s = check_epilogue(epilogue, dtype, y_dtype, n_out, &ep);
  if (s != SPLR_OK) return s;
  return run_fused(
      fused_call(X, M, n_in, nullptr, 1, values, meta, n_out, U, V, r, dtype, ep, Y, y_dtype, workspace), ws_bytes,
      stream);
}

size_t splr_linear_experts_workspace_bytes(int64_t M, int64_t n_experts, int64_t n_out, int64_t n_in, int64_t r,
                                           splr_dtype_t dtype) {
  return n_experts < 1 ? 0 : query_workspace_bytes(M, n_experts, n_out, n_in, r, dtype);
}

splr_status_t splr_linear_experts(const void* X, int64_t M, int64_t n_in, const int32_t* offsets, int64_t n_experts,
                                  const void* values, const uint32_t* meta, int64_t n_out, const void* U,
                                  const void* V, int64_t r, splr_dtype_t dtype, const splr_epilogue_t* epilogue,
                                  splr_dtype_t y_dtype, void* Y, void* workspace, size_t ws_bytes,
                                  hipStream_t stream) {
  if (!offsets || !values || !meta || (r > 0 && (!U || !V))) return SPLR_ERR_NULL;
  if (M != 0 && (!X || !Y)) return SPLR_ERR_NULL;
  splr_status_t s = check_in(n_in);
  if (s == SPLR_OK && (M < 0 || n_experts < 1 || n_experts > SPLR_EXPERTS_MAX)) s = SPLR_ERR_SHAPE;
  if (s == SPLR_OK && M > 0) s = check_rows(M, n_in);
  if (s == SPLR_OK) s = check_rows(n_out, n_in);
  if (s == SPLR_OK && n_experts * n_out * n_in > kMaxElems) s = SPLR_ERR_SHAPE;
  if (s == SPLR_OK) s = check_rank(r);
  if (s == SPLR_OK && M * n_out > kMaxElems) s = SPLR_ERR_SHAPE;
  if (s != SPLR_OK) return s;
  if (!dtype_ok(dtype)) return SPLR_ERR_DTYPE;
  splr::Epilogue ep;
  s = check_epilogue(epilogue, dtype, y_dtype, n_out, &ep);
  if (s != SPLR_OK) return s;
  if (!aligned16(X) || !aligned16(values) || !aligned16(meta) || !aligned16(Y) ||
      (reinterpret_cast<uintptr_t>(offsets) & 3u) || (r > 0 && (!aligned16(U) || !aligned16(V))))
    return SPLR_ERR_ALIGN;
  if (M == 0) return SPLR_OK;
  return run_fused(
      fused_call(X, M, n_in, offsets, n_experts, values, meta, n_out, U, V, r, dtype, ep, Y, y_dtype, workspace),
      ws_bytes, stream);
}

}  // extern "C"

// ---------------------------------------------------------------- tokens to experts and back
namespace {

constexpr int64_t kMaxSlots = int64_t(1) << 28;  // T slots

struct Span {
  const void* p;
  size_t bytes;
  bool meets(const Span& o) const {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(o.p);
    return p && o.p && bytes && o.bytes && (a < b ? b - a < bytes : a - b < o.bytes);
  }
};

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

splr_status_t check_slots(int64_t T, int64_t slots) {
  return T >= 0 && T < kMaxRows && slots >= 1 && slots <= SPLR_SLOTS_MAX && T * slots <= kMaxSlots ? SPLR_OK : SPLR_ERR_SHAPE;
}
// T rows of D entries, and `rows` rows of them
splr_status_t check_token_rows(int64_t T, int64_t rows, int64_t D, int size) {
  if (rows < 0 || rows > kMaxSlots || D < 1 || D > kMaxCols || T * D > kMaxElems || rows * D > kMaxElems) return SPLR_ERR_SHAPE;
  return splr::tokens_grids_fit(T, D, size) ? SPLR_OK : SPLR_ERR_SHAPE;
}
int entry_bytes(splr_dtype_t dtype) { return dtype == SPLR_FP32 ? 4 : dtype == SPLR_BF16 ? 2 : 1; }

}  // namespace

extern "C" {

size_t splr_tokens_dispatch_workspace_bytes(int64_t T, int64_t slots, int64_t n_experts) {
  if (check_slots(T, slots) != SPLR_OK || n_experts < 1 || n_experts > SPLR_EXPERTS_MAX) return 0;
  return round_up(splr::tokens_sort_workspace_bytes(T * slots, n_experts), 256);
}

splr_status_t splr_tokens_dispatch(const void* ids, int32_t id_bytes, int64_t T, int64_t slots, int64_t n_experts,
                                   const void* X, int64_t D, splr_dtype_t dtype, int32_t* offsets, int32_t* positions,
                                   void* Xs, void* workspace, size_t ws_bytes, hipStream_t stream) {
  if (!offsets || (T != 0 && (!ids || !positions)) || (T != 0 && !X != !Xs)) return SPLR_ERR_NULL;
  splr_status_t s = check_slots(T, slots);
  if (s == SPLR_OK && (n_experts < 1 || n_experts > SPLR_EXPERTS_MAX)) s = SPLR_ERR_SHAPE;
  if (s != SPLR_OK) return s;
  const bool copy = X && Xs;
  if (id_bytes != 4 && id_bytes != 8) return SPLR_ERR_DTYPE;
  if (copy && !dtype_ok(dtype) && dtype != SPLR_E4M3) return SPLR_ERR_DTYPE;
  const int size = entry_bytes(dtype);
  const int64_t N = T * slots;
  if (copy && (s = check_token_rows(T, N, D, size)) != SPLR_OK) return s;
  if ((reinterpret_cast<uintptr_t>(ids) & (id_bytes - 1)) || !aligned4(offsets) || !aligned4(positions) ||
      (copy && (!aligned16(X) || !aligned16(Xs))))
    return SPLR_ERR_ALIGN;
  const size_t need = splr_tokens_dispatch_workspace_bytes(T, slots, n_experts);
  if (need > 0 && (!workspace || ws_bytes < need)) return SPLR_ERR_WORKSPACE;
  if (need > 0 && !aligned16(workspace)) return SPLR_ERR_ALIGN;
  const Span out[] = {{offsets, (size_t)(n_experts + 1) * 4}, {positions, (size_t)N * 4},
                      {copy ? Xs : nullptr, (size_t)N * D * size}, {workspace, need}};
  const Span in[] = {{ids, (size_t)N * id_bytes}, {copy ? X : nullptr, (size_t)T * D * size}};
  for (int i = 0; i < 4; ++i) {
    for (const Span& x : in)
      if (out[i].meets(x)) return SPLR_ERR_OVERLAP;
    for (int j = 0; j < i; ++j)
      if (out[i].meets(out[j])) return SPLR_ERR_OVERLAP;
  }
  return from_hip(splr::launch_tokens_dispatch(ids, id_bytes == 8, T, slots, n_experts, offsets, positions, workspace,
                                               copy ? X : nullptr, D, size, Xs, stream));
}

splr_status_t splr_tokens_gather(const void* X, int64_t T, int64_t D, splr_dtype_t dtype, const int32_t* positions,
                                 int64_t slots, void* Xs, int64_t rows, hipStream_t stream) {
  if (T != 0 && (!X || !positions || (rows != 0 && !Xs))) return SPLR_ERR_NULL;
  splr_status_t s = check_slots(T, slots);
  if (s != SPLR_OK) return s;
  if (!dtype_ok(dtype) && dtype != SPLR_E4M3) return SPLR_ERR_DTYPE;
  const int size = entry_bytes(dtype);
  if ((s = check_token_rows(T, rows, D, size)) != SPLR_OK) return s;
  if (!aligned16(X) || !aligned4(positions) || !aligned16(Xs)) return SPLR_ERR_ALIGN;
  const Span out{Xs, (size_t)rows * D * size};
  if (out.meets({X, (size_t)T * D * size}) || out.meets({positions, (size_t)(T * slots) * 4})) return SPLR_ERR_OVERLAP;
  if (T == 0 || rows == 0) return SPLR_OK;
  return from_hip(splr::launch_tokens_gather(X, T, D, size, positions, slots, Xs, rows, stream));
}

splr_status_t splr_tokens_combine(const void* Z, int64_t rows, int64_t D, splr_dtype_t dtype, const int32_t* positions,
                                  int64_t T, int64_t slots, const float* weights, const void* residual, void* Y,
                                  hipStream_t stream) {
  if (T != 0 && ((rows != 0 && !Z) || !positions || !Y)) return SPLR_ERR_NULL;
  splr_status_t s = check_slots(T, slots);
  if (s != SPLR_OK) return s;
  if (!dtype_ok(dtype)) return SPLR_ERR_DTYPE;
  const int size = entry_bytes(dtype);
  if ((s = check_token_rows(T, rows, D, size)) != SPLR_OK) return s;
  if (!aligned16(Z) || !aligned4(positions) || !aligned4(weights) || !aligned16(residual) || !aligned16(Y)) return SPLR_ERR_ALIGN;
  const size_t row = (size_t)D * size, N = (size_t)(T * slots);
  const Span out{Y, (size_t)T * row};
  if (out.meets({Z, (size_t)rows * row}) || out.meets({positions, N * 4}) || out.meets({weights, N * 4}) ||
      (residual != Y && out.meets({residual, (size_t)T * row})))
    return SPLR_ERR_OVERLAP;
  if (T == 0) return SPLR_OK;
  return from_hip(splr::launch_tokens_combine(Z, rows, D, dtype == SPLR_BF16, positions, T, slots, weights, residual, Y, stream));
}

splr_status_t splr_tokens_combine_backward(const void* dY, const void* Z, int64_t rows, int64_t D, splr_dtype_t dtype,
                                           const int32_t* positions, int64_t T, int64_t slots, const float* weights, void* dZ,
                                           float* dweights, hipStream_t stream) {
  if (T != 0 && (!dY || !positions || (!dZ && !dweights && rows != 0) || (dweights && rows != 0 && !Z))) return SPLR_ERR_NULL;
  splr_status_t s = check_slots(T, slots);
  if (s != SPLR_OK) return s;
  if (!dtype_ok(dtype)) return SPLR_ERR_DTYPE;
  const int size = entry_bytes(dtype);
  if ((s = check_token_rows(T, rows, D, size)) != SPLR_OK) return s;
  if (!aligned16(dY) || !aligned16(Z) || !aligned4(positions) || !aligned4(weights) || !aligned16(dZ) || !aligned4(dweights))
    return SPLR_ERR_ALIGN;
  const size_t row = (size_t)D * size, N = (size_t)(T * slots);
  const Span dz{dZ, (size_t)rows * row}, dw{dweights, N * 4}, z{dweights ? Z : nullptr, (size_t)rows * row};
  const Span in[] = {{dY, (size_t)T * row}, {positions, N * 4}, {weights, N * 4}};
  for (const Span& x : in)
    if (dz.meets(x) || dw.meets(x)) return SPLR_ERR_OVERLAP;
  if (dz.meets(dw) || dw.meets(z) || (dZ != Z && dz.meets(z))) return SPLR_ERR_OVERLAP;
  if (T == 0 || (!dZ && !dweights)) return SPLR_OK;
  return from_hip(splr::launch_tokens_combine_backward(dY, Z, rows, D, dtype == SPLR_BF16, positions, T, slots, weights, dZ,
                                                       dweights, stream));
}

// ---------------------------------------------------------------- weights in 8 bits

splr_status_t splr_fp8_quantize(const void* X, int64_t rows, int64_t cols, splr_dtype_t dtype, int32_t block_rows,
                                int32_t transposed, void* Q, float* scales, hipStream_t stream) {
  if (!X || !Q || !scales) return SPLR_ERR_NULL;
  if (rows < 1 || cols < 1 || rows > kMaxRows || cols > kMaxRows || rows * cols > kMaxElems) return SPLR_ERR_SHAPE;
  // Q's rows are the products' reduction dimension
  if (transposed ? rows > kMaxCols : (cols % 32 != 0 || cols > kMaxCols)) return SPLR_ERR_SHAPE;
  if (block_rows != 1 && block_rows != 128) return SPLR_ERR_SHAPE;
  if (!dtype_ok(dtype)) return SPLR_ERR_DTYPE;
  const bool block = block_rows == 128;
  if (!splr::fp8_quantize_grids_fit(rows, cols, block, transposed != 0)) return SPLR_ERR_SHAPE;
  if (!aligned16(X) || !aligned16(Q) || !aligned4(scales)) return SPLR_ERR_ALIGN;
  const size_t R = (size_t)rows, C = (size_t)cols, rb = (R + 127) / 128, cb = (C + 127) / 128;
  const Span x{X, R * C * entry_bytes(dtype)}, q{Q, transposed ? C * ((R + 31) / 32 * 32) : R * C},
      sc{scales, 4 * (block ? rb * cb : transposed ? rb * C : R * cb)};
  if (x.meets(q) || x.meets(sc) || q.meets(sc)) return SPLR_ERR_OVERLAP;
  return from_hip(splr::launch_fp8_quantize(X, rows, cols, dtype == SPLR_BF16, block, transposed != 0, Q, scales, stream));
}

}  // extern "C"

namespace {

bool x_type_ok(splr_dtype_t dtype) { return dtype_ok(dtype) || dtype == SPLR_E4M3; }

// The checks of both products; n_experts 0: one layer. c gets the call.
splr_status_t check_fp8(const void* X, const float* x_scales, int64_t M, int64_t n_in, splr_dtype_t dtype,
                        const int32_t* offsets, int64_t n_experts, const void* W, const float* w_scales, int32_t w_block_rows,
                        int64_t n_out, const splr_epilogue_t* epilogue, splr_dtype_t y_dtype, void* Y, void* workspace,
                        splr::Fp8Call* c) {
  const bool experts = n_experts != 0, rows = M != 0 || !experts;
  if (!W || !w_scales || (rows && (!X || !Y || (dtype == SPLR_E4M3 && !x_scales)))) return SPLR_ERR_NULL;
  splr_status_t s = check_in(n_in);
  if (s == SPLR_OK && (M < 0 || n_experts < 0 || n_experts > SPLR_EXPERTS_MAX)) s = SPLR_ERR_SHAPE;
  if (s == SPLR_OK && rows) s = check_rows(M, n_in);
  if (s == SPLR_OK) s = check_rows(n_out, n_in);
  const int64_t E = experts ? n_experts : 1;
  if (s == SPLR_OK && (E * n_out * n_in > kMaxElems || M * n_out > kMaxElems)) s = SPLR_ERR_SHAPE;
  if (s == SPLR_OK && w_block_rows != 1 && w_block_rows != 128) s = SPLR_ERR_SHAPE;
  if (s != SPLR_OK) return s;
  if (!x_type_ok(dtype)) return SPLR_ERR_DTYPE;
  splr::Epilogue ep;
  s = check_epilogue(epilogue, y_dtype, y_dtype, n_out, &ep);
  if (s != SPLR_OK) return s;
  if (!aligned16(X) || !aligned16(W) || !aligned16(Y) || !aligned4(x_scales) || !aligned4(w_scales) || !aligned4(offsets))
    return SPLR_ERR_ALIGN;
  *c = splr::Fp8Call{X, (int)dtype, dtype == SPLR_E4M3 ? x_scales : nullptr, M, n_in, offsets, E, (const uint8_t*)W, w_scales,
                     w_block_rows == 1, n_out, ep, Y, y_dtype == SPLR_BF16, workspace};
  return SPLR_OK;
}

splr_status_t run_fp8(const splr::Fp8Call& c, size_t ws_bytes, hipStream_t stream) {
  splr::Fp8Plan plan;
  if (!splr::plan_fp8(c, &plan)) return SPLR_ERR_SHAPE;
  const size_t need = round_up(splr::fp8_workspace_bytes(c, plan), 256);
  if (need > 0 && (!c.workspace || ws_bytes < need)) return SPLR_ERR_WORKSPACE;
  if (need > 0 && !aligned16(c.workspace)) return SPLR_ERR_ALIGN;
  const size_t E = (size_t)c.experts, M = (size_t)c.M, n_in = (size_t)c.n_in, n_out = (size_t)c.n_out;
  const size_t KB = (n_in + 127) / 128, y_size = c.y_bf16 ? 2 : 4;
  const Span y{c.Y, M * n_out * y_size}, workspace{c.workspace, need};
  const Span read[] = {{c.X, M * n_in * entry_bytes((splr_dtype_t)c.x_type)},
                       {c.x_scales, M * KB * 4},
                       {c.offsets, (E + 1) * 4},
                       {c.W, E * n_out * n_in},
                       {c.w_scales, E * KB * (c.w_rows ? n_out : (n_out + 127) / 128) * 4},
                       {c.ep.bias, E * n_out * y_size}};
  for (const Span& x : read)
    if (y.meets(x) || workspace.meets(x)) return SPLR_ERR_OVERLAP;
  for (const void* p : {c.ep.gate, c.ep.residual})
    if (workspace.meets({p, y.bytes}) || (p != c.Y && y.meets({p, y.bytes}))) return SPLR_ERR_OVERLAP;
  if (workspace.meets(y)) return SPLR_ERR_OVERLAP;
  return from_hip(splr::launch_fp8(c, plan, stream));
}

// A call by its sizes and its plan, for the queries; false when it would be refused or has no rows. n_experts 0: one layer.
bool query_fp8(int64_t M, int64_t n_experts, int64_t n_out, int64_t n_in, splr_dtype_t dtype, splr_dtype_t y_dtype,
               splr::Fp8Call* c, splr::Fp8Plan* plan) {
  if (M < 1 || M > kMaxRows || n_out < 1 || n_out > splr::kMaxFusedOut || n_experts < 0 || n_experts > SPLR_EXPERTS_MAX ||
      check_in(n_in) != SPLR_OK || !x_type_ok(dtype) || !dtype_ok(y_dtype))
    return false;
  static const int32_t any = 0;  // a non-null `offsets`: a call by expert
  *c = splr::Fp8Call{nullptr, (int)dtype, nullptr, M, n_in, n_experts ? &any : nullptr, n_experts ? n_experts : 1, nullptr,
                     nullptr, false, n_out, splr::Epilogue{}, nullptr, y_dtype == SPLR_BF16, nullptr};
  return splr::plan_fp8(*c, plan);
}

}  // namespace

extern "C" {

size_t splr_linear_fp8_workspace_bytes(int64_t M, int64_t n_experts, int64_t n_out, int64_t n_in, splr_dtype_t dtype,
                                       splr_dtype_t y_dtype) {
  splr::Fp8Call c;
  splr::Fp8Plan plan;
  return query_fp8(M, n_experts, n_out, n_in, dtype, y_dtype, &c, &plan) ? round_up(splr::fp8_workspace_bytes(c, plan), 256) : 0;
}

splr_status_t splr_linear_fp8_tile(int64_t M, int64_t n_experts, int64_t n_out, int64_t n_in, splr_dtype_t dtype,
                                   splr_dtype_t y_dtype, int32_t* rows, int32_t* tokens) {
  if (!rows || !tokens) return SPLR_ERR_NULL;
  splr::Fp8Call c;
  splr::Fp8Plan plan;
  if (!query_fp8(M, n_experts, n_out, n_in, dtype, y_dtype, &c, &plan)) return SPLR_ERR_SHAPE;
  *rows = plan.rows;
  *tokens = plan.tokens;
  return SPLR_OK;
}

splr_status_t splr_linear_fp8(const void* X, const float* x_scales, int64_t M, int64_t n_in, splr_dtype_t dtype, const void* W,
                              const float* w_scales, int32_t w_block_rows, int64_t n_out, const splr_epilogue_t* epilogue,
                              splr_dtype_t y_dtype, void* Y, void* workspace, size_t ws_bytes, hipStream_t stream) {
  splr::Fp8Call c;
  const splr_status_t s = check_fp8(X, x_scales, M, n_in, dtype, nullptr, 0, W, w_scales, w_block_rows, n_out, epilogue, y_dtype,
                                    Y, workspace, &c);
  return s != SPLR_OK ? s : run_fp8(c, ws_bytes, stream);
}

splr_status_t splr_linear_fp8_experts(const void* X, const float* x_scales, int64_t M, int64_t n_in, splr_dtype_t dtype,
                                      const int32_t* offsets, int64_t n_experts, const void* W, const float* w_scales,
                                      int32_t w_block_rows, int64_t n_out, const splr_epilogue_t* epilogue,
                                      splr_dtype_t y_dtype, void* Y, void* workspace, size_t ws_bytes, hipStream_t stream) {
  if (!offsets) return SPLR_ERR_NULL;
  if (n_experts < 1) return SPLR_ERR_SHAPE;
  splr::Fp8Call c;
  const splr_status_t s = check_fp8(X, x_scales, M, n_in, dtype, offsets, n_experts, W, w_scales, w_block_rows, n_out, epilogue,
                                    y_dtype, Y, workspace, &c);
  if (s != SPLR_OK) return s;
  return M == 0 ? SPLR_OK : run_fp8(c, ws_bytes, stream);
}

}  // extern "C"

// ---------------------------------------------------------------- splr_linear_noalloc
// For callers that cannot allocate: the first-stage workspace lives in a file-scope device array.
// Each GPU the library runs on holds its own copy (from the first call on it until the process
// ends), at its own address, found once per device with hipGetSymbolAddress. In host code the
// array's name is only a stand-in for the symbol; kernels get the looked-up device address.
namespace {

constexpr size_t kScratchBytes = size_t(32) << 20;  // SPLR_LINEAR_NOALLOC_MAX_WORKSPACE in splr.h
static_assert(kScratchBytes == SPLR_LINEAR_NOALLOC_MAX_WORKSPACE, "header and library agree");
__device__ __align__(256) uint8_t scratch[kScratchBytes];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices];

// This device's copy of `scratch`, looked up on the first call with that device current.
hipError_t device_scratch(void** out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (!g_scratch_ptr[dev]) {
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (e != hipSuccess) return e;
    if (!p) return hipErrorInvalidSymbol;
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return hipSuccess;
}

}  // namespace

extern "C" {

splr_status_t splr_linear_noalloc(const void* X, int64_t M, int64_t n_in, const void* values, const uint32_t* meta,
                                  int64_t n_out, const void* U, const void* V, int64_t r, splr_dtype_t dtype, float* Y,
                                  hipStream_t stream) {
  const splr_status_t s =
      check_linear(X, M, n_in, values, meta, n_out, U, V, r, dtype, Y, nullptr, 0, true, true, false);
  if (s != SPLR_OK) return s;
  const size_t need = workspace_bytes(M, n_in, r, dtype);
  if (need > kScratchBytes) return SPLR_ERR_SCRATCH;
  void* ws = nullptr;
  if (need > 0 && device_scratch(&ws) != hipSuccess) return SPLR_ERR_HIP;
  // the same kernels as splr_linear; the workspace needs no clearing (every byte the second stage
  // reads is written by the first stage of this call)
  if (splr::launch_lowrank(X, V, M, n_in, r, dtype == SPLR_BF16, ws, stream) != hipSuccess) return SPLR_ERR_HIP;
  return run_stage2(X, M, n_in, values, meta, n_out, U, r, dtype, Y, false, ws, stream);
}

splr_status_t splr_dense_reconstruct(const void* values, const uint32_t* meta, const void* U, const void* V,
                                     int64_t n_out, int64_t n_in, int64_t r, splr_dtype_t dtype, float* W_hat,
                                     hipStream_t stream) {
  if (!values || !meta || !W_hat) return SPLR_ERR_NULL;
  if (r > 0 && (!U || !V)) return SPLR_ERR_NULL;
  splr_status_t s = check_in(n_in);
  if (s == SPLR_OK) s = check_rows(n_out, n_in);
  if (s == SPLR_OK) s = check_rank(r);
  if (s != SPLR_OK) return s;
  if (!dtype_ok(dtype)) return SPLR_ERR_DTYPE;
  if (!splr::reconstruct_grids_fit(n_out, n_in)) return SPLR_ERR_SHAPE;
  if (!aligned16(values) || !aligned16(meta) || !aligned16(W_hat)) return SPLR_ERR_ALIGN;
  if (r > 0 && (!aligned16(U) || !aligned16(V))) return SPLR_ERR_ALIGN;
  return from_hip(splr::launch_dense_reconstruct(values, meta, U, V, n_out, n_in, r, dtype == SPLR_BF16, W_hat,
                                                 stream));
}

size_t splr_gram_workspace_bytes(int64_t n, int64_t k) {
  if (n < 1 || n > kMaxCols || k < 1 || k > splr::kMaxCholK) return 0;
  return round_up(splr::gram_workspace_bytes(n, k), 256);
}

splr_status_t splr_gram_f64(const float* Y, int64_t n, int64_t k, double* G, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
  if (!Y || !G) return SPLR_ERR_NULL;
  if (n < 1 || n > kMaxCols || k < 1 || k > splr::kMaxCholK) return SPLR_ERR_SHAPE;
  if (!workspace || workspace_bytes < splr_gram_workspace_bytes(n, k)) return SPLR_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(Y) & 3u) || (reinterpret_cast<uintptr_t>(G) & 7u) ||
      (reinterpret_cast<uintptr_t>(workspace) & 7u))
    return SPLR_ERR_ALIGN;
  return from_hip(splr::launch_gram_f64(Y, n, k, G, workspace, stream));
}

splr_status_t splr_chol_rinv(const double* G, int64_t k, float* Rinv, hipStream_t stream) {
  if (!G || !Rinv) return SPLR_ERR_NULL;
  if (k < 1 || k > splr::kMaxCholK) return SPLR_ERR_SHAPE;
  if ((reinterpret_cast<uintptr_t>(G) & 7u) || (reinterpret_cast<uintptr_t>(Rinv) & 3u)) return SPLR_ERR_ALIGN;
  return from_hip(splr::launch_chol_rinv(G, k, Rinv, stream));
}

const char* splr_status_string(splr_status_t status) {
  switch (status) {
    case SPLR_OK: return "SPLR_OK";
    case SPLR_ERR_NULL: return "SPLR_ERR_NULL: a required pointer is NULL";
    case SPLR_ERR_SHAPE: return "SPLR_ERR_SHAPE: a size is out of range";
    case SPLR_ERR_DTYPE: return "SPLR_ERR_DTYPE: unknown dtype";
    case SPLR_ERR_ALIGN: return "SPLR_ERR_ALIGN: a pointer is not 16-byte aligned";
    case SPLR_ERR_HIP: return "SPLR_ERR_HIP: the HIP runtime reported an error";
    case SPLR_ERR_WORKSPACE: return "SPLR_ERR_WORKSPACE: workspace missing or too small";
    case SPLR_ERR_SCRATCH:
      return "SPLR_ERR_SCRATCH: the call needs more workspace than splr_linear_noalloc's built-in buffer holds";
    case SPLR_ERR_OVERLAP: return "SPLR_ERR_OVERLAP: Y or the workspace overlaps another operand";
  }
  return "SPLR_ERR_UNKNOWN";
}

// The library version, followed by the first 16 hex digits of the SHA-256 of the sources it was
// built from (the build passes it in), so a loaded binary can be matched to a source tree.
#ifndef SPLR_SOURCE_SHA
#define SPLR_SOURCE_SHA "unknown"
#endif
const char* splr_version(void) { return "0.2.0+" SPLR_SOURCE_SHA; }

}  // extern "C"
