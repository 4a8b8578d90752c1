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

// An output in an input's place has its rows where the input's are, or a row written lies on rows still to be read.
domino_status check_in_place(const void* out, int64_t ld_out, const void* in, int64_t ld_in, int64_t rows, const char* what) {
  if (rows > 1 && in && out == in && ld_out != ld_in)
    return refuse(DOMINO_ERR_INVALID_ARG, std::string(what) + " share their memory with different row strides");
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

// Tensor map of a row-major rows x cols matrix with row stride ld (elements), a third dimension of one.
domino_status map2(CUtensorMap* m, int elem_bytes, const void* base, int64_t cols, int64_t rows, int64_t ld,
                   uint32_t box_cols, uint32_t box_rows, int swizzle) {
  const uint64_t dims[3] = {uint64_t(cols), uint64_t(rows), 1};
  const uint64_t strides[2] = {uint64_t(ld) * elem_bytes, uint64_t(ld) * uint64_t(rows) * elem_bytes};
  const uint32_t box[3] = {box_cols, box_rows, 1};
  std::string err;
  if (!dm::make_map(m, elem_bytes, base, 3, dims, strides, box, &err, swizzle)) return refuse(DOMINO_ERR_CUDA, err);
  return DOMINO_OK;
}

constexpr size_t kSlice = 1024;
size_t slice_up(size_t n) { return (n + kSlice - 1) / kSlice * kSlice; }

domino_status check_linear(int64_t m, int64_t n, int64_t k, int32_t act) {
  if (m < 0 || n <= 0 || k <= 0) return refuse(DOMINO_ERR_INVALID_ARG, "need M >= 0, N > 0 and K > 0");
  if (act < DOMINO_ACT_NONE || act > DOMINO_ACT_BILINEAR) return refuse(DOMINO_ERR_INVALID_ARG, "unknown activation");
  if (act > DOMINO_ACT_GELU)
    return refuse(DOMINO_ERR_UNSUPPORTED, "the linear layer takes no gated activation (domino_mlp_fwd does)");
  if (n % 8 != 0 || k % 8 != 0) return refuse(DOMINO_ERR_ALIGNMENT, "N and K must be multiples of 8 (16-byte rows)");
  if (m > (int64_t(1) << 31) - 257 || n > (int64_t(1) << 20) || k > (int64_t(1) << 20))
    return refuse(DOMINO_ERR_UNSUPPORTED, "linear layer: M beyond 2^31 - 257, or N or K beyond 2^20");
  if (((m + 255) / 256) * ((n + 255) / 256) >= int64_t(1) << 30)
    return refuse(DOMINO_ERR_UNSUPPORTED, "linear layer: more output tiles than one launch covers");
  return DOMINO_OK;
}

// Rows that one launch adds to gW_main: that kernel waits at most two seconds for a tile, whose 2^20 steps of 64 rows
// take 0.3.
constexpr int64_t kMainRows = int64_t(1) << 26;

// Workspace of the backward: gZ, and the bias gradient's partial sums.  gZ's rows begin at multiples of 128 bytes, so
// that a row of a TMA box is one line: with neither gZ nor the other operand so, the products of 4729 x 9032 and 9368
// columns take 556 and 550 us, with gZ 468 and 447.
int64_t gz_stride(int64_t n) { return (n + 63) / 64 * 64; }
struct LinBwdPlan {
  size_t off_gz, off_part, total;
};
LinBwdPlan linear_bwd_plan(int64_t m, int64_t n, int32_t act) {
  LinBwdPlan p = {};
  p.off_part = p.off_gz + (act == DOMINO_ACT_NONE ? 0 : slice_up(size_t(m) * gz_stride(n) * 2));
  p.total = p.off_part + slice_up(size_t(dm::lin_gz_row_blocks(m, n)) * n * 4);
  if (m == 0) p.total = 0;
  return p;
}

domino_status check_packed(int64_t tq, int64_t n, int32_t heads, int32_t kv_heads, int64_t tk) {
  if (tq < 0 || n < 0 || tk < 0 || heads < 1 || kv_heads < 1)
    return refuse(DOMINO_ERR_INVALID_ARG, "need tq, n, tk >= 0, heads >= 1 and kv_heads >= 1");
  if (heads % kv_heads != 0) return refuse(DOMINO_ERR_INVALID_ARG, "heads must be a multiple of kv_heads");
  if (heads / kv_heads > 128 || heads > 4096)
    return refuse(DOMINO_ERR_UNSUPPORTED, "packed attention: more than 128 heads per key head, or than 4096 heads");
  const int64_t most = (int64_t(1) << 31) - 1024;
  if (tq > most || tk > most || n > (int64_t(1) << 24) || (tq + n + 1024) * kv_heads > most)
    return refuse(DOMINO_ERR_UNSUPPORTED, "packed attention: more tokens or sequences than one call covers");
  return DOMINO_OK;
}

// Arguments and operand maps of D (m x n) = A . B^T over k: A m x k and B n x k, each contiguous along the
// reduction or (a_mn, b_mn) given as its transpose, with row strides ld_a, ld_b.
domino_status linear_product(dm::LinMaps* maps, dm::LinArgs* a, const uint16_t* A, int64_t ld_a, bool a_mn,
                             const uint16_t* B, int64_t ld_b, bool b_mn, int64_t m, int64_t n, int64_t k, int site) {
  const dm::LinPlan p = dm::lin_plan(m, n, k);
  *a = {};
  a->M = int32_t(m);
  a->N = int32_t(n);
  a->m_tiles = int32_t((m + 255) / 256);
  a->n_tiles = int32_t((n + p.width - 1) / p.width);
  a->k_blocks = int32_t((k + 63) / 64);
  a->err_site = site << 4;
  a->width = p.width;
  a->parts = p.parts;
  a->units = p.units;
  a->a_rows = a_mn || m >= 128 ? 128 : int32_t((m + 7) / 8 * 8);
  DM_TRY(a_mn ? map2(&maps->a, 2, A, m, k, ld_a, 64, 64, 128) : map2(&maps->a, 2, A, k, m, ld_a, 64, uint32_t(a->a_rows), 128));
  DM_TRY(b_mn ? map2(&maps->b, 2, B, n, k, ld_b, 64, 64, 128) : map2(&maps->b, 2, B, k, n, ld_b, 64, uint32_t(p.width / 2), 128));
  return DOMINO_OK;
}

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
      DM_TRY(check_in_place(Y, ld_y, X, ld_x, rows, "Y and X"));
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
      DM_TRY(check_in_place(gX, ld_gx, gY, ld_gy, rows, "gX and gY"));
      DM_TRY(check_in_place(gX, ld_gx, gres, ld_gres, rows, "gX and gres"));
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

domino_status domino_linear_bwd_workspace_size(int64_t M, int64_t N, int64_t K, int32_t act, size_t* bytes) {
  return guarded([&]() -> domino_status {
    if (!bytes) return refuse(DOMINO_ERR_INVALID_ARG, "bytes is NULL");
    DM_TRY(check_linear(M, N, K, act));
    *bytes = linear_bwd_plan(M, N, act).total;
    return DOMINO_OK;
  });
}

domino_status domino_linear_fwd(domino_handle H, const uint16_t* X, int64_t ld_x, const uint16_t* W,
                                const uint16_t* bias, int32_t act, const uint16_t* R, int64_t ld_r, uint16_t* Y,
                                int64_t ld_y, uint16_t* Z, int64_t ld_z, int64_t M, int64_t N, int64_t K,
                                void* stream) {
  return guarded([&]() -> domino_status {
    DM_TRY(check_linear(M, N, K, act));
    DM_TRY(check_ld(ld_x, K, "ld_x"));
    DM_TRY(check_ld(ld_y, N, "ld_y"));
    if (R) DM_TRY(check_ld(ld_r, N, "ld_r"));
    if (Z) DM_TRY(check_ld(ld_z, N, "ld_z"));
    DM_TRY(check_ptr(W, "W"));
    DM_TRY(check_ptr(bias, "bias", true));
    if (M > 0) {
      DM_TRY(check_ptr(X, "X"));
      DM_TRY(check_ptr(Y, "Y"));
      DM_TRY(check_ptr(R, "R", true));
      DM_TRY(check_ptr(Z, "Z", true));
      DM_TRY(check_in_place(Y, ld_y, R, ld_r, M, "Y and R"));
    }
    DM_TRY(dm::check_handle(H));
    if (M == 0) return DOMINO_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (M <= dm::kFewRows) {
      dm::LinFewArgs a = {};
      a.M = int32_t(M);
      a.N = int32_t(N);
      a.act = act;
      a.err_site = 0x24 << 4;
      a.bias = bias;
      a.R = R;
      a.Y = Y;
      a.Z = Z;
      a.ld_r = ld_r;
      a.ld_y = ld_y;
      a.ld_z = ld_z;
      dm::lin_few_plan(M, N, K, &a);
      CUtensorMap w, x;
      DM_TRY(map2(&w, 2, W, K, N, K, 64, uint32_t(a.height), 128));
      DM_TRY(map2(&x, 2, X, K, M, ld_x, 64, uint32_t(a.x_rows), 128));
      return dm::launch_on(H, DOMINO_K_LINEAR_FWD, st, "linear layer launch (few rows)",
                           [&] { return dm::launch_linear_few(w, x, a, st); });
    }
    dm::LinMaps m = {};
    dm::LinArgs a;
    DM_TRY(linear_product(&m, &a, X, ld_x, false, W, K, false, M, N, K, 0x20));
    DM_TRY(map2(&m.y, 2, Y, N, M, ld_y, 32, 32, 64));
    if (Z) DM_TRY(map2(&m.z, 2, Z, N, M, ld_z, 32, 32, 64));
    a.act = act;
    a.save = Z != nullptr;
    a.bias = bias;
    a.R = R;
    a.ld_r = ld_r;
    return dm::launch_on(H, DOMINO_K_LINEAR_FWD, st, "linear layer launch",
                         [&] { return dm::launch_linear(dm::LIN_FWD, m, a, st); });
  });
}

domino_status domino_linear_bwd(domino_handle H, const uint16_t* gY, int64_t ld_gy, const uint16_t* X, int64_t ld_x,
                                const uint16_t* W, const uint16_t* Z, int64_t ld_z, int32_t act, uint16_t* gX,
                                int64_t ld_gx, uint16_t* gW, float* gW_main, float* gbias, int32_t accumulate,
                                int64_t M, int64_t N, int64_t K, void* workspace, size_t workspace_bytes,
                                void* stream) {
  return guarded([&]() -> domino_status {
    DM_TRY(check_linear(M, N, K, act));
    if (accumulate != 0 && accumulate != 1) return refuse(DOMINO_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    if (gW && gW_main) return refuse(DOMINO_ERR_INVALID_ARG, "gW and gW_main exclude each other");
    DM_TRY(check_ld(ld_gy, N, "ld_gy"));
    const bool want_gw = gW || gW_main, has_act = act != DOMINO_ACT_NONE;
    if (want_gw) DM_TRY(check_ld(ld_x, K, "ld_x"));
    if (gX) DM_TRY(check_ld(ld_gx, K, "ld_gx"));
    if (has_act) DM_TRY(check_ld(ld_z, N, "ld_z"));
    DM_TRY(check_ptr(gW, "gW", true));
    DM_TRY(check_ptr(gW_main, "gW_main", true));
    DM_TRY(check_ptr(gbias, "gbias", true));
    const LinBwdPlan P = linear_bwd_plan(M, N, act);
    if (M > 0) {
      DM_TRY(check_ptr(gY, "gY"));
      DM_TRY(check_ptr(gX, "gX", true));
      if (want_gw) DM_TRY(check_ptr(X, "X"));
      if (gX) DM_TRY(check_ptr(W, "W"));
      if (has_act) DM_TRY(check_ptr(Z, "Z"));
      DM_TRY(check_ws(workspace, workspace_bytes, P.total));
    }
    DM_TRY(dm::check_handle(H));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (M == 0) {  // empty sums
      if (gW && cudaMemsetAsync(gW, 0, size_t(N) * K * 2, st) != cudaSuccess)
        return refuse(DOMINO_ERR_CUDA, "cudaMemsetAsync failed");
      if (gbias && !accumulate && cudaMemsetAsync(gbias, 0, size_t(N) * 4, st) != cudaSuccess)
        return refuse(DOMINO_ERR_CUDA, "cudaMemsetAsync failed");
      return DOMINO_OK;
    }
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    uint16_t* gz_buf = reinterpret_cast<uint16_t*>(ws + P.off_gz);
    float* part = reinterpret_cast<float*>(ws + P.off_part);
    if (has_act || gbias) {
      const dm::LinGzArgs g = {gY, Z, gz_buf, gbias ? part : nullptr, M, N, ld_gy, ld_z, gz_stride(N), act};
      DM_TRY(dm::launch_on(H, DOMINO_K_LINEAR_GZ, st, "linear layer gZ launch", [&] { return dm::launch_lin_gz(g, st); }));
      if (gbias)
        DM_TRY(dm::launch_on(H, DOMINO_K_LINEAR_GZ, st, "linear layer bias gradient launch",
                             [&] { return dm::launch_lin_gbias(part, M, N, gbias, accumulate, st); }));
    }
    const uint16_t* gZ = has_act ? gz_buf : gY;
    const int64_t ld_gz = has_act ? gz_stride(N) : ld_gy;
    if (gX) {
      dm::LinMaps m = {};
      dm::LinArgs a;
      DM_TRY(linear_product(&m, &a, gZ, ld_gz, false, W, K, true, M, K, N, 0x21));
      DM_TRY(map2(&m.y, 2, gX, K, M, ld_gx, 32, 32, 64));
      DM_TRY(dm::launch_on(H, DOMINO_K_LINEAR_GX, st, "linear layer gX launch",
                           [&] { return dm::launch_linear(dm::LIN_GX, m, a, st); }));
    }
    if (gW) {
      dm::LinMaps m = {};
      dm::LinArgs a;
      DM_TRY(linear_product(&m, &a, gZ, ld_gz, true, X, ld_x, true, N, K, M, 0x22));
      DM_TRY(map2(&m.y, 2, gW, K, N, K, 32, 32, 64));
      DM_TRY(dm::launch_on(H, DOMINO_K_LINEAR_GW, st, "linear layer gW launch",
                           [&] { return dm::launch_linear(dm::LIN_GW, m, a, st); }));
    }
    // gW_main: the MLP's weight-gradient product, tiles of 256 x 256, added up over ranges of rows
    for (int64_t r = 0; gW_main && r < M; r += kMainRows) {
      dm::LinMaps m = {};
      dm::LinArgs a;
      DM_TRY(linear_product(&m, &a, gZ + r * ld_gz, ld_gz, true, X + r * ld_x, ld_x, true, N, K, M - r < kMainRows ? M - r : kMainRows, 0x22));
      dm::GemmArgs g = {};
      g.batches = 1;
      g.m_tiles = a.m_tiles;
      g.n_tiles = int32_t((K + 255) / 256);
      g.k_blocks = a.k_blocks;
      g.M = a.M;
      g.N = a.N;
      g.err_site = a.err_site;
      g.alpha = g.out_scale = 1.0f;
      g.out0 = gW_main;
      g.ld0 = K;
      const dm::EpiMaps none = {};
      DM_TRY(dm::launch_on(H, DOMINO_K_LINEAR_GW, st, "linear layer gW launch",
                           [&] { return dm::launch_gemm_bwd(dm::GV_WGRAD, m.a, m.b, none, g, st); }));
    }
    return DOMINO_OK;
  });
}

domino_status domino_attn_packed_workspace_size(int64_t tq, int64_t n, int32_t heads, int32_t kv_heads, int64_t tk,
                                                size_t* bytes) {
  return guarded([&]() -> domino_status {
    if (!bytes) return refuse(DOMINO_ERR_INVALID_ARG, "bytes is NULL");
    DM_TRY(check_packed(tq, n, heads, kv_heads, tk));
    *bytes = tq == 0 || n == 0 ? 0 : size_t(dm::packed_scratch_bytes(tq, n, heads, kv_heads, tk));
    return DOMINO_OK;
  });
}

domino_status domino_attn_packed_fwd(domino_handle H, const uint16_t* Q, int64_t ld_q, const uint16_t* K, int64_t ld_k,
                                     const uint16_t* V, int64_t ld_v, const int32_t* cu_q, const int32_t* k_start,
                                     const int32_t* k_len, float scale, uint16_t* O, int64_t ld_o, float* lse,
                                     int64_t tq, int64_t n, int32_t heads, int32_t kv_heads, int64_t tk,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  return guarded([&]() -> domino_status {
    DM_TRY(check_packed(tq, n, heads, kv_heads, tk));
    if (!(scale > 0.0f) || !std::isfinite(scale * 1.4426950408889634f))
      return refuse(DOMINO_ERR_INVALID_ARG, "scale must be > 0, and finite in base 2 (at most 2.3e38)");
    DM_TRY(check_ld(ld_q, int64_t(heads) * 128, "ld_q"));
    DM_TRY(check_ld(ld_k, int64_t(kv_heads) * 128, "ld_k"));
    DM_TRY(check_ld(ld_v, int64_t(kv_heads) * 128, "ld_v"));
    DM_TRY(check_ld(ld_o, int64_t(heads) * 128, "ld_o"));
    const bool work = tq > 0 && n > 0;
    if (work) {
      DM_TRY(check_ptr(Q, "Q"));
      DM_TRY(check_ptr(K, "K", tk == 0));
      DM_TRY(check_ptr(V, "V", tk == 0));
      DM_TRY(check_ptr(O, "O"));
      DM_TRY(check_ptr(lse, "lse", true));
      const int32_t* lists[] = {cu_q, k_start, k_len};
      static const char* const names[] = {"cu_q", "k_start", "k_len"};
      for (int i = 0; i < 3; ++i) {
        if (!lists[i]) return refuse(DOMINO_ERR_INVALID_ARG, std::string(names[i]) + " is NULL");
        if (reinterpret_cast<uintptr_t>(lists[i]) & 3u)
          return refuse(DOMINO_ERR_ALIGNMENT, std::string(names[i]) + " is not 4-byte aligned");
      }
      DM_TRY(check_ws(workspace, workspace_bytes, size_t(dm::packed_scratch_bytes(tq, n, heads, kv_heads, tk))));
    }
    DM_TRY(dm::check_handle(H));
    if (!work) return DOMINO_OK;
    dm::PackedArgs a = {};
    a.cu_q = cu_q;
    a.k_start = k_start;
    a.k_len = k_len;
    a.O = O;
    a.lse = lse;
    a.ld_o = ld_o;
    a.n = int32_t(n);
    a.tq = int32_t(tq);
    a.tk = int32_t(tk);
    a.hq = heads;
    a.hkv = kv_heads;
    a.group = heads / kv_heads;
    a.tokens = 128 / a.group;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.scale_two = std::ldexp(1.0f, std::ilogb(a.scale_log2));
    a.raise_by = 8.0f / a.scale_log2;
    a.huge = 0x1p28f / a.scale_log2;
    a.err_site = 0x23 << 4;
    dm::packed_groups(&a, op_sms(H));
    std::string err;
    CUtensorMap mq, mk, mv;
    {
      const uint64_t dims[4] = {128, uint64_t(a.group), uint64_t(kv_heads), uint64_t(tq)};
      const uint64_t strides[3] = {256, uint64_t(a.group) * 256, uint64_t(ld_q) * 2};
      const uint32_t box[4] = {64, uint32_t(a.group), 1, uint32_t(a.tokens)};
      if (!dm::make_map(&mq, 2, Q, 4, dims, strides, box, &err)) return refuse(DOMINO_ERR_CUDA, err);
    }
    for (int i = 0; i < 2; ++i) {
      // without keys nothing is loaded: the maps describe Q's first row
      const uint64_t dims[3] = {128, uint64_t(kv_heads), uint64_t(tk > 0 ? tk : 1)};
      const uint64_t strides[2] = {256, uint64_t(i ? ld_v : ld_k) * 2};
      const uint32_t box[3] = {64, 1, 128};
      if (!dm::make_map(i ? &mv : &mk, 2, tk > 0 ? (i ? V : K) : Q, 3, dims, strides, box, &err))
        return refuse(DOMINO_ERR_CUDA, err);
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    DM_TRY(dm::launch_on(H, DOMINO_K_ATTN_PACKED, st, "packed attention plan launch",
                         [&] { return dm::launch_packed_plan(a, workspace, st); }));
    DM_TRY(dm::launch_on(H, DOMINO_K_ATTN_PACKED, st, "packed attention launch",
                         [&] { return dm::launch_packed_attention(mq, mk, mv, a, workspace, st); }));
    if (dm::packed_may_cut(a))
      DM_TRY(dm::launch_on(H, DOMINO_K_ATTN_PACKED, st, "packed attention combine launch",
                           [&] { return dm::launch_packed_combine(a, workspace, st); }));
    return DOMINO_OK;
  });
}

}  // extern "C"
