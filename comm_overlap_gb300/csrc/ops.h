// ops.h -- host-side interface between the C ABI of the sublayer operators (ops_api.cu) and their
// kernels: LayerNorm with parameters (norm.cu), the linear layer (linear.cu),
// attention over packed sequences (packed_attention.cu), norms and rotation of queries and keys and the
// 8-bit cache (rotary.cu), attention over that cache (cached_attention.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <functional>
#include <string>
#include <utility>

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

// ---- programmatic dependent launch: a kernel may be placed on SMs that its predecessor in the stream has left, and
// sets itself up there; before it touches memory that others use it waits, in every thread's path, for the
// predecessor's end (pdl_wait).  Saves 2 - 3 us between the short kernels of these operators.  The predecessor writes
// while the kernel already runs, so no memory is read-only for the kernel's lifetime: such kernels read with ordinary
// loads after the wait, never through __ldg, ld.global.nc or pointers declared __restrict__, which a compiler may move
// before it.
#ifdef __CUDACC__
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

template <class... Params, class... Args>
cudaError_t launch_pdl(void (*fn)(Params...), dim3 grid, dim3 block, size_t smem, int cluster, cudaStream_t st,
                       Args&&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fn, static_cast<Params>(std::forward<Args>(args))...);
}
#endif

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
cudaError_t take_norm_error(int* code);
cudaError_t launch_ln_cols(const LnBwdArgs& a, const float* part, int sms, cudaStream_t st);

// ---- linear layer (linear.cu): D (M x N) = A . B^T over k_blocks steps of 64
constexpr int kLinPairs = 76;  // CTA pairs of a GB300; more are not used
enum LinKind : int {
  LIN_FWD = 0,  // A, B contiguous along the reduction: X . W^T
  LIN_GX = 1,   // B contiguous along its rows: gZ . W
  LIN_GW = 2,   // both contiguous along their rows: gZ^T . X
};
// How a product is laid over the GPU: tiles of 256 x width, each computed by `parts` pairs along the
// reduction, by `units` pairs (groups of `parts` pairs).
struct LinPlan {
  int width, parts, units;
};
LinPlan lin_plan(int64_t m, int64_t n, int64_t k);
// Maps (all with a third dimension of one): operands in boxes of 64 (reduction) x a_rows, or x width / 2 for
// B, or, contiguous along their rows, 64 (rows) x 64 (reduction), 128-byte swizzle; y, z (z only with save) in
// boxes of 32 x 32, 64-byte swizzle.
struct LinMaps {
  CUtensorMap a, b, y, z;
};
struct LinArgs {
  int32_t M, N, m_tiles, n_tiles, k_blocks, act, save, err_site;
  int32_t width, parts, units;  // lin_plan
  int32_t a_rows;               // rows of a box of A: 128, or fewer when A is smaller
  int32_t stages, stage_bytes;  // set by the launcher: the operand ring
  const uint16_t* bias;         // nullable
  const uint16_t* R;            // nullable
  int64_t ld_r;
};
cudaError_t launch_linear(int kind, const LinMaps& m, LinArgs a, cudaStream_t st);
// The layer on few rows (at most kFewRows): tiles of `height` rows of W, split along the reduction over `parts` CTAs of a
// cluster, by `units` clusters.  Maps (third dimension of one, 128-byte swizzle): w in boxes of 64 x height, x in
// boxes of 64 x x_rows.
constexpr int kFewRows = 64;
struct LinFewArgs {
  int32_t M, N, k_blocks, act, err_site;
  int32_t height, parts, tiles, units, x_rows;  // lin_few_plan
  int32_t stages, stage_bytes;                  // set by the launcher: the operand ring
  const uint16_t* bias;                         // nullable
  const uint16_t* R;                            // nullable
  uint16_t* Y;
  uint16_t* Z;                                  // nullable
  int64_t ld_r, ld_y, ld_z;
};
void lin_few_plan(int64_t m, int64_t n, int64_t k, LinFewArgs* a);
cudaError_t launch_linear_few(const CUtensorMap& w, const CUtensorMap& x, LinFewArgs a, cudaStream_t st);
struct LinGzArgs {
  const uint16_t* gY;
  const uint16_t* Z;  // with an activation
  uint16_t* gZ;       // with an activation
  float* part;        // nullable: lin_gz_row_blocks() rows of N floats
  int64_t M, N, ld_gy, ld_z, ld_gz;
  int32_t act;
};
int lin_gz_row_blocks(int64_t m, int64_t n);
cudaError_t launch_lin_gz(const LinGzArgs& a, cudaStream_t st);
cudaError_t launch_lin_gbias(const float* part, int64_t m, int64_t n, float* gbias, int accumulate, cudaStream_t st);
cudaError_t take_linear_error(int* code);

// ---- causal attention over packed sequences (packed_attention.cu), head dimension 128
constexpr int kPackedMinPart = 4;          // key blocks of 128 in the smallest part of a cut item
constexpr int kPackedBadLengths = 0x7E0;   // error word: a sequence's rows leave the tensors
struct PackedArgs {
  const int32_t* cu_q;     // n + 1
  const int32_t* k_start;  // n
  const int32_t* k_len;    // n
  uint16_t* O;
  float* lse;              // nullable: tq x hq
  int64_t ld_o;
  int32_t n, tq, tk, hq, hkv, group, tokens;  // group = hq / hkv query heads share a key head; tokens = 128 / group
  int32_t heads_abreast, subgroups, groups;   // packed_groups: key heads of a group of CTAs, hkv / that, groups
  float scale_log2;        // scale x log2(e)
  float scale_two;         // the power of two below it
  float raise_by, huge;    // scores: 8 and 2^28 over scale_log2
  int32_t err_site;
};
// Maps, bf16 with 128-byte swizzle: q (128, group, hkv, tq) in boxes (64, group, 1, tokens); k, v (128, hkv,
// tk) in boxes (64, 1, 128).
int64_t packed_scratch_bytes(int64_t tq, int64_t n, int hq, int hkv, int64_t tk);
void packed_groups(PackedArgs* a, int sms);
bool packed_may_cut(const PackedArgs& a);
cudaError_t launch_packed_plan(const PackedArgs& a, void* ws, cudaStream_t st);
cudaError_t launch_packed_attention(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                    const PackedArgs& a, void* ws, cudaStream_t st);
cudaError_t launch_packed_combine(const PackedArgs& a, void* ws, cudaStream_t st);
cudaError_t take_packed_error(int* code);

// ---- norm and rotation of query and key heads, the 8-bit cache (rotary.cu), head dimension 128
constexpr int kCacheExpMax = 51;  // the cache's powers of two lie between 2^-51 and 2^51
struct RotaryArgs {
  const uint16_t* Q;
  const uint16_t* K;            // nullable with hkv = 0
  const uint16_t* V;            // into the cache
  const int32_t* positions;     // with rot > 0
  const double* frequencies;    // with rot > 0: rot / 2, radians a position
  const uint16_t* wq;           // nullable: no norm
  const uint16_t* wk;
  uint16_t* Yq;
  uint16_t* Yk;                 // not into the cache
  uint8_t* k8;                  // nullable: the cache, rows x hkv x 128 codes, and hkv rows of exponents + 127
  uint8_t* v8;
  uint8_t* k_exp;
  uint8_t* v_exp;
  const int32_t* rows;          // the cache row of each token; negative: not written
  int64_t tokens, ld_q, ld_k, ld_v, ld_yq, ld_yk, ld_exp;
  int32_t hq, hkv, rot, layout, cache_rows;  // layout: 0 half, 1 interleaved
  float eps, amplitude, sign;   // sign -1: rotated back
};
struct RotaryBwdArgs {
  const uint16_t* gYq;
  const uint16_t* gYk;
  const uint16_t* Q;
  const uint16_t* K;
  const int32_t* positions;
  const double* frequencies;
  const uint16_t* wq;
  const uint16_t* wk;
  uint16_t* gQ;
  uint16_t* gK;
  float* gwq;
  float* gwk;                   // nullable with hkv = 0
  int64_t tokens, ld_gyq, ld_gyk, ld_q, ld_k, ld_gq, ld_gk;
  int32_t hq, hkv, rot, layout, accumulate;
  float eps, amplitude;
};
struct CacheReadArgs {
  const uint8_t* k8;
  const uint8_t* v8;
  const uint8_t* k_exp;
  const uint8_t* v_exp;
  const int32_t* rows;          // negative: zeros
  uint16_t* K;
  uint16_t* V;
  int64_t tokens, ld_k, ld_v, ld_exp;
  int32_t hkv, cache_rows;
};
cudaError_t launch_rotary(const RotaryArgs& a, int sms, cudaStream_t st);
// `part`: rotary_bwd_blocks() rows of 128 floats, written by the backward and summed by launch_rotary_sums.
int rotary_bwd_blocks(int64_t tokens, int hq, int hkv, int sms);
cudaError_t launch_rotary_bwd(const RotaryBwdArgs& a, float* part, int sms, cudaStream_t st);
cudaError_t launch_rotary_sums(const RotaryBwdArgs& a, const float* part, int sms, cudaStream_t st);
cudaError_t launch_cache_read(const CacheReadArgs& a, int sms, cudaStream_t st);
cudaError_t take_rotary_error(int* code);

// ---- attention of the last tokens of each sequence over the 8-bit cache (cached_attention.cu)
struct CachedArgs {
  const uint16_t* Q;
  const uint8_t* k_exp;
  const uint8_t* v_exp;
  const int32_t* k_start;  // n
  const int32_t* k_len;    // n
  uint16_t* O;
  float* lse;              // nullable
  int64_t ld_q, ld_o, ld_exp;
  const int32_t* prefix;                 // nullable: first row and number of the rows that all sequences see
  int64_t whole_rows;                    // cached_shape, as the next two lines: n x t x hq
  int32_t rows, rows_of_block, blocks;   // rows (tokens x group) of a sequence and key head, in blocks
  int32_t shared_rows, shared_blocks;    // those of all sequences together, over the shared rows
  int32_t abreast;                       // neighbouring key heads that blocks take at the same time
  int32_t n, t, hq, hkv, group, cache_rows, shared;  // query i of t sees k_len - t + i + 1 keys; shared: 1 with a prefix
  float scale_log2;                      // scale x log2(e)
};
// Maps of codes, 128-byte swizzle: (128, hkv, cache_rows) in boxes (128, 1, kCachedKeys).
constexpr int kCachedKeys = 128;
void cached_shape(CachedArgs* a);
int64_t cached_scratch_bytes(const CachedArgs& a);
cudaError_t launch_cached_attention(const CUtensorMap& k, const CUtensorMap& v, const CachedArgs& a, void* ws, int sms, cudaStream_t st);
cudaError_t launch_cached_join(const CachedArgs& a, void* ws, cudaStream_t st);
cudaError_t take_cached_error(int* code);

}  // namespace dm
