// ops_api.cu -- the C ABI of the sublayer operators (include/domino.h): argument validation,
// workspace layout and launches.
#include <cmath>
#include <new>

#include "ops.h"

namespace {

// Workspaces are sized for the SMs of a GB300 (a size query has no device to ask); launchers cap
// their grids by the same number, so a device with more SMs leaves some idle instead of overrunning.
constexpr int kGb300Sms = 152;

domino_status refuse(domino_status s, const std::string& msg) {
  dm::set_last_error(msg);
  return s;
}

// No C++ exception leaves an entry point.
template <class Fn>
domino_status guarded(Fn&& fn) {
  try {
    return fn();
  } catch (const std::bad_alloc&) {
    return DOMINO_ERR_CUDA;
  } catch (...) {
    return DOMINO_ERR_CUDA;
  }
}

#define DM_TRY(expr)                 \
  do {                               \
    const domino_status s_ = (expr); \
    if (s_ != DOMINO_OK) return s_;  \
  } while (0)

domino_status check_ptr(const void* p, const char* name, bool nullable = false) {
  if (!p) return nullable ? DOMINO_OK : refuse(DOMINO_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) & 15u)
    return refuse(DOMINO_ERR_ALIGNMENT, std::string(name) + " is not 16-byte aligned");
  return DOMINO_OK;
}

domino_status check_ld(int64_t ld, int64_t cols, const char* name) {
  if (ld < cols) return refuse(DOMINO_ERR_INVALID_ARG, std::string(name) + " is smaller than the row it strides over");
  if (ld % 8 != 0) return refuse(DOMINO_ERR_ALIGNMENT, std::string(name) + " must be a multiple of 8 (16-byte rows)");
  if (ld > (int64_t(1) << 32)) return refuse(DOMINO_ERR_UNSUPPORTED, std::string(name) + " beyond the supported range");
  return DOMINO_OK;
}

domino_status check_ws(void* ws, size_t bytes, size_t need) {
  if (need == 0) return DOMINO_OK;
  if (!ws) return refuse(DOMINO_ERR_WORKSPACE, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(ws) & 255u) return refuse(DOMINO_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  if (bytes < need)
    return refuse(DOMINO_ERR_WORKSPACE, "workspace too small: need " + std::to_string(need) + " bytes");
  return DOMINO_OK;
}

int op_sms(domino_handle H) {
  const int n = dm::handle_sms(H);
  return n < kGb300Sms ? n : kGb300Sms;
}

domino_status check_ln(int64_t rows, int64_t h) {
  if (rows < 0 || h <= 0) return refuse(DOMINO_ERR_INVALID_ARG, "need rows >= 0 and h > 0");
  if (h % 8 != 0) return refuse(DOMINO_ERR_ALIGNMENT, "h must be a multiple of 8 (16-byte rows)");
  if (h > dm::kLnMaxH || rows > (int64_t(1) << 31) - 1)
    return refuse(DOMINO_ERR_UNSUPPORTED, "LayerNorm: h beyond 16384 or rows beyond 2^31 - 1");
  return DOMINO_OK;
}

size_t ln_bwd_bytes(int64_t rows, int64_t h) { return size_t(dm::ln_bwd_blocks(rows, h, kGb300Sms)) * 2 * h * 4; }

}  // namespace

extern "C" {

domino_status domino_layernorm_fwd(domino_handle H, const uint16_t* X, int64_t ld_x, const uint16_t* gamma,
                                   const uint16_t* beta, float eps, uint16_t* Y, int64_t ld_y, float* mean,
                                   float* rstd, int64_t rows, int64_t h, void* stream) {
  return guarded([&]() -> domino_status {
    DM_TRY(check_ln(rows, h));
    if (!(eps > 0.0f) || !std::isfinite(eps)) return refuse(DOMINO_ERR_INVALID_ARG, "eps must be finite and > 0");
    DM_TRY(check_ld(ld_x, h, "ld_x"));
    DM_TRY(check_ld(ld_y, h, "ld_y"));
    if (rows > 0) {
      DM_TRY(check_ptr(X, "X"));
      DM_TRY(check_ptr(gamma, "gamma"));
      DM_TRY(check_ptr(beta, "beta", true));
      DM_TRY(check_ptr(Y, "Y"));
      DM_TRY(check_ptr(mean, "mean", true));
      DM_TRY(check_ptr(rstd, "rstd", true));
    }
    DM_TRY(dm::check_handle(H));
    if (rows == 0) return DOMINO_OK;
    const dm::LnFwdArgs a = {X, gamma, beta, Y, mean, rstd, rows, h, ld_x, ld_y, eps};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dm::launch_on(H, DOMINO_K_LN_AFFINE, st, "LayerNorm launch",
                         [&] { return dm::launch_ln_fwd(a, op_sms(H), st); });
  });
}

domino_status domino_layernorm_bwd_workspace_size(int64_t rows, int64_t h, size_t* bytes) {
  return guarded([&]() -> domino_status {
    if (!bytes) return refuse(DOMINO_ERR_INVALID_ARG, "bytes is NULL");
    DM_TRY(check_ln(rows, h));
    *bytes = ln_bwd_bytes(rows, h);
    return DOMINO_OK;
  });
}

domino_status domino_layernorm_bwd(domino_handle H, const uint16_t* gY, int64_t ld_gy, const uint16_t* X,
                                   int64_t ld_x, const uint16_t* gamma, const float* mean, const float* rstd,
                                   const uint16_t* gres, int64_t ld_gres, uint16_t* gX, int64_t ld_gx, float* ggamma,
                                   float* gbeta, int32_t accumulate, int64_t rows, int64_t h, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  return guarded([&]() -> domino_status {
    DM_TRY(check_ln(rows, h));
    if (accumulate != 0 && accumulate != 1) return refuse(DOMINO_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    DM_TRY(check_ld(ld_gy, h, "ld_gy"));
    DM_TRY(check_ld(ld_x, h, "ld_x"));
    DM_TRY(check_ld(ld_gx, h, "ld_gx"));
    if (gres) DM_TRY(check_ld(ld_gres, h, "ld_gres"));
    DM_TRY(check_ptr(gamma, "gamma"));
    DM_TRY(check_ptr(ggamma, "ggamma"));
    DM_TRY(check_ptr(gbeta, "gbeta", true));
    if (rows > 0) {
      DM_TRY(check_ptr(gY, "gY"));
      DM_TRY(check_ptr(X, "X"));
      DM_TRY(check_ptr(mean, "mean"));
      DM_TRY(check_ptr(rstd, "rstd"));
      DM_TRY(check_ptr(gres, "gres", true));
      DM_TRY(check_ptr(gX, "gX"));
    }
    DM_TRY(check_ws(workspace, workspace_bytes, ln_bwd_bytes(rows, h)));
    DM_TRY(dm::check_handle(H));
    const dm::LnBwdArgs a = {gY, X, gamma, mean, rstd, gres, gX, ggamma, gbeta, rows, h, ld_gy, ld_x, ld_gres, ld_gx,
                             accumulate};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    float* part = static_cast<float*>(workspace);
    if (rows > 0)
      DM_TRY(dm::launch_on(H, DOMINO_K_LN_AFFINE_BWD, st, "LayerNorm backward launch",
                           [&] { return dm::launch_ln_bwd(a, part, op_sms(H), st); }));
    return dm::launch_on(H, DOMINO_K_LN_AFFINE_BWD, st, "LayerNorm gradient sums launch",
                         [&] { return dm::launch_ln_cols(a, part, op_sms(H), st); });
  });
}

}  // extern "C"
