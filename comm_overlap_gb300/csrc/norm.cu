// norm.cu -- LayerNorm with weight and bias, forward and backward with the reduction of the weight's
// and bias's gradients over the rows.
//
// A team of `tpr` threads (whole warps) holds one row at a time: thread i owns the 16-byte pieces i,
// i + tpr, ... (NPT of them) of every row it sees, so each input is read from memory once, the two
// passes of the forward run in registers, and the backward keeps its columns' sums of the weight and
// bias gradients in registers over all rows of the team.  Teams walk the rows with a fixed stride;
// the next row's pieces are loaded before the current row is reduced, which keeps memory busy across
// the reductions.  All arithmetic is fp32; the one rounding to bf16 is the output's.
// Bound: memory (forward 4 bytes, backward 6, with a residual gradient 8 bytes an element).
#include "actfn.cuh"
#include "ops.h"

namespace dm {

namespace {

constexpr int kTeamThreads = 512;  // widest team, and the widest block

// Sums of a and b over the team, the same bits in every thread: warp butterflies, then the warps'
// sums in warp order.  `red`: 2 x 16 pairs of this team, alternating (`flip`), so that one barrier
// separates a sum's writes from its reads and the next-but-one sum's writes from both.
__device__ __forceinline__ float2 team_sum(float a, float b, float2* red, int& flip, int warps, int team) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
  }
  if (warps == 1) return make_float2(a, b);
  float2* r = red + 16 * flip;
  flip ^= 1;
  const int wt = (threadIdx.x >> 5) - team * warps;
  if ((threadIdx.x & 31) == 0) r[wt] = make_float2(a, b);
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(warps * 32) : "memory");
  float2 s = r[0];
  for (int w = 1; w < warps; ++w) {
    s.x += r[w].x;
    s.y += r[w].y;
  }
  return s;
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  v[0] = bf16lo(w.x); v[1] = bf16hi(w.x); v[2] = bf16lo(w.y); v[3] = bf16hi(w.y);
  v[4] = bf16lo(w.z); v[5] = bf16hi(w.z); v[6] = bf16lo(w.w); v[7] = bf16hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

template <int NPT>
__device__ __forceinline__ void load_row(uint4 (&w)[NPT], const uint16_t* p, int t, int tpr, int nv) {
  const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
  for (int i = 0; i < NPT; ++i) {
    const int v = t + i * tpr;
    w[i] = v < nv ? __ldcs(q + v) : make_uint4(0u, 0u, 0u, 0u);
  }
}

// mean and 1 / sqrt(var + eps) of the row (variance of the centred values, as a second pass over the
// registers), y = (x - mean) rstd gamma + beta.
template <int NPT>
__global__ void __launch_bounds__(kTeamThreads) ln_fwd_kernel(const LnFwdArgs a, const int tpr) {
  pdl_launch();
  pdl_wait();
  __shared__ float2 red_all[8][32];
  const int team = threadIdx.x / tpr, t = threadIdx.x - team * tpr, warps = tpr >> 5;
  const int teams = blockDim.x / tpr;
  const int nv = static_cast<int>(a.h >> 3);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * teams;
  int64_t r = static_cast<int64_t>(blockIdx.x) * teams + team;
  if (r >= a.rows) return;
  float2* red = red_all[team];
  int flip = 0;
  const float inv_h = 1.0f / static_cast<float>(a.h);
  uint4 w[NPT], ga[NPT], be[NPT];
  load_row<NPT>(w, a.X + r * a.ld_x, t, tpr, nv);
#pragma unroll
  for (int i = 0; i < NPT; ++i) {
    const int v = t + i * tpr;
    ga[i] = v < nv ? reinterpret_cast<const uint4*>(a.gamma)[v] : make_uint4(0u, 0u, 0u, 0u);
    be[i] = v < nv && a.beta ? reinterpret_cast<const uint4*>(a.beta)[v] : make_uint4(0u, 0u, 0u, 0u);
  }
  for (; r < a.rows; r += stride) {
    uint4 next[NPT];
    const bool more = r + stride < a.rows;
    if (more) load_row<NPT>(next, a.X + (r + stride) * a.ld_x, t, tpr, nv);
    // mean and variance of the row times c
    auto stats = [&](float c, float& mean, float& var) {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < NPT; ++i) {
        float x[8];
        unpack8(w[i], x);  // pieces past the row are zero
        s += ((x[0] * c + x[1] * c) + (x[2] * c + x[3] * c)) + ((x[4] * c + x[5] * c) + (x[6] * c + x[7] * c));
      }
      mean = team_sum(s, 0.0f, red, flip, warps, team).x * inv_h;
      float q = 0.0f;
#pragma unroll
      for (int i = 0; i < NPT; ++i) {
        if (t + i * tpr >= nv) continue;
        float x[8];
        unpack8(w[i], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(x[e] * c - mean, x[e] * c - mean, q);
      }
      var = team_sum(q, 0.0f, red, flip, warps, team).x * inv_h;
    };
    float c = 1.0f, mean, var;
    stats(1.0f, mean, var);
    if (!(var < INFINITY)) {  // the squares' sum left fp32's range (or the row holds an infinity or NaN)
      c = 0x1p-80f;
      stats(c, mean, var);
    }
    const float rstd = 1.0f / sqrtf(var + a.eps * c * c);
    if (t == 0) {
      if (a.mean) a.mean[r] = mean / c;
      if (a.rstd) a.rstd[r] = rstd * c;
    }
    uint4* y = reinterpret_cast<uint4*>(a.Y + r * a.ld_y);
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
      if (t + i * tpr >= nv) continue;
      float x[8], g[8], b[8];
      unpack8(w[i], x);
      unpack8(ga[i], g);
      unpack8(be[i], b);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf((x[e] * c - mean) * rstd, g[e], b[e]);
      y[t + i * tpr] = pack8(x);
    }
    if (more) {
#pragma unroll
      for (int i = 0; i < NPT; ++i) w[i] = next[i];
    }
  }
}

// With u = gy gamma and n = (x - mean) rstd:  gx = rstd (u - mean(u) - n mean(u n)) (+ gres);
// the columns' sums of gy n and gy over the block's rows go to row blockIdx.x of `part` (2 h floats).
template <int NPT, bool PREFETCH>
__global__ void __launch_bounds__(kTeamThreads) ln_bwd_kernel(const LnBwdArgs a, float* __restrict__ part,
                                                              const int tpr) {
  extern __shared__ float cols[];  // teams x 2 h (only with several teams)
  pdl_launch();
  pdl_wait();
  __shared__ float2 red_all[8][32];
  const int team = threadIdx.x / tpr, t = threadIdx.x - team * tpr, warps = tpr >> 5;
  const int teams = blockDim.x / tpr;
  const int nv = static_cast<int>(a.h >> 3);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * teams;
  int64_t r = static_cast<int64_t>(blockIdx.x) * teams + team;
  float2* red = red_all[team];
  int flip = 0;
  const float inv_h = 1.0f / static_cast<float>(a.h);
  float ag[NPT][8], ab[NPT][8];
  uint4 ga[NPT], gw[NPT], xw[NPT];
  // the widest rows leave no registers for gamma and the next row: both are then loaded where used
  const uint4* gp = reinterpret_cast<const uint4*>(a.gamma);
  auto gamma_at = [&](int i) {
    const int v = t + i * tpr;
    return v < nv ? gp[v] : make_uint4(0u, 0u, 0u, 0u);
  };
#pragma unroll
  for (int i = 0; i < NPT; ++i) {
    if constexpr (PREFETCH) ga[i] = gamma_at(i);
#pragma unroll
    for (int e = 0; e < 8; ++e) ag[i][e] = ab[i][e] = 0.0f;
  }
  float mean = 0.0f, rstd = 0.0f;
  if (PREFETCH && r < a.rows) {
    load_row<NPT>(gw, a.gY + r * a.ld_gy, t, tpr, nv);
    load_row<NPT>(xw, a.X + r * a.ld_x, t, tpr, nv);
    mean = a.mean[r];
    rstd = a.rstd[r];
  }
  for (; r < a.rows; r += stride) {
    uint4 ng[NPT], nx[NPT], rw[NPT];
    if constexpr (!PREFETCH) {
      load_row<NPT>(gw, a.gY + r * a.ld_gy, t, tpr, nv);
      load_row<NPT>(xw, a.X + r * a.ld_x, t, tpr, nv);
      mean = a.mean[r];
      rstd = a.rstd[r];
    }
    float nmean = 0.0f, nrstd = 0.0f;
    const int64_t rn = r + stride;
    const bool more = rn < a.rows;
    if constexpr (PREFETCH) {
      if (a.gres) load_row<NPT>(rw, a.gres + r * a.ld_gres, t, tpr, nv);
      if (more) {
        load_row<NPT>(ng, a.gY + rn * a.ld_gy, t, tpr, nv);
        load_row<NPT>(nx, a.X + rn * a.ld_x, t, tpr, nv);
        nmean = a.mean[rn];
        nrstd = a.rstd[rn];
      }
    }
    float su = 0.0f, sun = 0.0f;
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
      float g[8], x[8], m[8];
      unpack8(gw[i], g);  // zero past the row
      unpack8(xw[i], x);
      unpack8(PREFETCH ? ga[i] : gamma_at(i), m);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = (x[e] - mean) * rstd, u = g[e] * m[e];
        su += u;
        sun = fmaf(u, n, sun);
        ag[i][e] = fmaf(g[e], n, ag[i][e]);
        ab[i][e] += g[e];
      }
    }
    const float2 s = team_sum(su, sun, red, flip, warps, team);
    const float mu = s.x * inv_h, mun = s.y * inv_h;
    uint4* o = reinterpret_cast<uint4*>(a.gX + r * a.ld_gx);
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
      if (t + i * tpr >= nv) continue;
      float g[8], x[8], m[8], z[8];
      unpack8(gw[i], g);
      unpack8(xw[i], x);
      unpack8(PREFETCH ? ga[i] : gamma_at(i), m);
      if (a.gres)
        unpack8(PREFETCH ? rw[i] : __ldcs(reinterpret_cast<const uint4*>(a.gres + r * a.ld_gres) + t + i * tpr), z);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = (x[e] - mean) * rstd, u = g[e] * m[e];
        x[e] = fmaf(rstd, u - mu - n * mun, z[e]);
      }
      o[t + i * tpr] = pack8(x);
    }
    if constexpr (PREFETCH) {
      if (more) {
#pragma unroll
        for (int i = 0; i < NPT; ++i) {
          gw[i] = ng[i];
          xw[i] = nx[i];
        }
        mean = nmean;
        rstd = nrstd;
      }
    }
  }
  float* out = part + static_cast<int64_t>(blockIdx.x) * 2 * a.h;
  if (teams == 1) {
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
      const int c = (t + i * tpr) * 8;
      if (c >= a.h) continue;
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        *reinterpret_cast<float4*>(out + c + e) = make_float4(ag[i][e], ag[i][e + 1], ag[i][e + 2], ag[i][e + 3]);
        *reinterpret_cast<float4*>(out + a.h + c + e) = make_float4(ab[i][e], ab[i][e + 1], ab[i][e + 2], ab[i][e + 3]);
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NPT; ++i) {
    const int c = (t + i * tpr) * 8;
    if (c >= a.h) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cols[team * 2 * a.h + c + e] = ag[i][e];
      cols[team * 2 * a.h + a.h + c + e] = ab[i][e];
    }
  }
  __syncthreads();
  for (int64_t c = threadIdx.x; c < 2 * a.h; c += blockDim.x) {
    float s = cols[c];
    for (int k = 1; k < teams; ++k) s += cols[k * 2 * a.h + c];
    out[c] = s;
  }
}

// Column sums of `parts` rows of 2 h floats, in a fixed order: 32 groups of rows per block, then the
// groups in order.  Columns 0 .. h-1 go to ggamma, the others to gbeta (nullable).
__global__ void __launch_bounds__(1024) ln_cols_kernel(const float* __restrict__ part, int parts, int64_t h,
                                                       float* ggamma, float* gbeta, int accumulate) {
  pdl_launch();
  pdl_wait();
  __shared__ float4 sums[32][32];
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * 32 + lane) * 4;
  const bool in = c < 2 * h;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (in) {
#pragma unroll 4
    for (int p = grp; p < parts; p += 32) {
      const float4 v = *reinterpret_cast<const float4*>(part + p * 2 * h + c);
      s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
  }
  sums[grp][lane] = s;
  __syncthreads();
  if (grp != 0 || !in) return;
  for (int k = 1; k < 32; ++k) {
    const float4 v = sums[k][lane];
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  float* o = c < h ? ggamma + c : (gbeta ? gbeta + (c - h) : nullptr);  // h % 8 == 0: never straddles
  if (!o) return;
  if (accumulate) {
    const float4 v = *reinterpret_cast<const float4*>(o);
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  *reinterpret_cast<float4*>(o) = s;
}

int pieces_per_thread(int64_t h) { return h <= 2048 ? 1 : (h <= 8192 ? 2 : 4); }
int team_threads(int64_t h, int npt) { return static_cast<int>(((h / 8 + npt - 1) / npt + 31) / 32 * 32); }

}  // namespace

int ln_bwd_blocks(int64_t rows, int64_t h, int sms) {
  const int tpr = team_threads(h, pieces_per_thread(h)), teams = tpr >= 256 ? 1 : 256 / tpr;
  const int64_t need = (rows + 4 * teams - 1) / (4 * teams), most = 2 * int64_t(sms);
  return static_cast<int>(need < most ? need : most);
}

cudaError_t launch_ln_fwd(const LnFwdArgs& a, int sms, cudaStream_t st) {
  if (a.rows == 0) return cudaSuccess;
  const int npt = pieces_per_thread(a.h), tpr = team_threads(a.h, npt), teams = tpr >= 256 ? 1 : 256 / tpr;
  const int64_t need = (a.rows + teams - 1) / teams, most = int64_t(sms) * (2048 / (teams * tpr));
  const dim3 grid(static_cast<unsigned>(need < most ? need : most)), block(static_cast<unsigned>(teams * tpr));
  return launch_pdl(npt == 1 ? ln_fwd_kernel<1> : npt == 2 ? ln_fwd_kernel<2> : ln_fwd_kernel<4>, grid, block, 0, 1, st, a, tpr);
}

cudaError_t launch_ln_bwd(const LnBwdArgs& a, float* part, int sms, cudaStream_t st) {
  const int grid = ln_bwd_blocks(a.rows, a.h, sms);
  if (grid == 0) return cudaSuccess;
  const int npt = pieces_per_thread(a.h), tpr = team_threads(a.h, npt), teams = tpr >= 256 ? 1 : 256 / tpr;
  // several teams only for h <= 1024 (at most 8 teams x 2 h floats with teams x h <= 2048)
  const size_t smem = teams > 1 ? size_t(teams) * 2 * a.h * 4 : 0;
  return launch_pdl(npt == 1 ? ln_bwd_kernel<1, true> : npt == 2 ? ln_bwd_kernel<2, true> : ln_bwd_kernel<4, false>, dim3(grid),
                    dim3(static_cast<unsigned>(teams * tpr)), smem, 1, st, a, part, tpr);
}

cudaError_t launch_ln_cols(const LnBwdArgs& a, const float* part, int sms, cudaStream_t st) {
  const int grid = ln_bwd_blocks(a.rows, a.h, sms);
  const int cgrid = static_cast<int>((2 * a.h + 127) / 128);
  return launch_pdl(ln_cols_kernel, dim3(cgrid), dim3(1024), 0, 1, st, part, grid, a.h, a.ggamma, a.gbeta, a.accumulate);
}

}  // namespace dm
