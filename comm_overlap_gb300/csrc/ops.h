// ops.h -- host-side interface between the C ABI of the sublayer operators (ops_api.cu) and their
// kernels: LayerNorm with parameters (norm.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <functional>
#include <string>

#include "../../include/domino.h"
#include "kernels.h"

namespace dm {

// ---- what api.cu shares with the other translation units of the C ABI
void set_last_error(const std::string& msg);
domino_status check_handle(domino_handle H);  // non-null and bound to the current device
int handle_sms(domino_handle H);
// One launch through the handle: launch count, per-kernel timing, failure injection, NVTX range.
domino_status launch_on(domino_handle H, int kind, cudaStream_t st, const char* what,
                        const std::function<cudaError_t()>& fn);

// ---- LayerNorm with weight and bias (norm.cu); h a multiple of 8, at most kLnMaxH
constexpr int64_t kLnMaxH = 16384;
struct LnFwdArgs {
  const uint16_t* X;
  const uint16_t* gamma;
  const uint16_t* beta;  // nullable
  uint16_t* Y;
  float* mean;  // nullable
  float* rstd;  // nullable
  int64_t rows, h, ld_x, ld_y;
  float eps;
};
struct LnBwdArgs {
  const uint16_t* gY;
  const uint16_t* X;
  const uint16_t* gamma;
  const float* mean;
  const float* rstd;
  const uint16_t* gres;  // nullable
  uint16_t* gX;
  float* ggamma;
  float* gbeta;  // nullable
  int64_t rows, h, ld_gy, ld_x, ld_gres, ld_gx;
  int32_t accumulate;
};
cudaError_t launch_ln_fwd(const LnFwdArgs& a, int sms, cudaStream_t st);
// `part`: ln_bwd_blocks() rows of 2 h floats, written by the backward and summed by launch_ln_cols.
int ln_bwd_blocks(int64_t rows, int64_t h, int sms);
cudaError_t launch_ln_bwd(const LnBwdArgs& a, float* part, int sms, cudaStream_t st);
cudaError_t launch_ln_cols(const LnBwdArgs& a, const float* part, int sms, cudaStream_t st);

}  // namespace dm
