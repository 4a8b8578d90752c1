// norm.cu -- LayerNorm with weight and bias, forward and backward with the reduction of the weight's
// and bias's gradients over the rows.
//
// A team of `tpr` threads (whole warps) holds one row at a time: thread i owns the 16-byte pieces i,
// i + tpr, ... (NPT of them) of every row it sees, so each input is read from memory once, the two
// passes of the forward run in registers, and the backward keeps its columns' sums of the weight and
// bias gradients in registers over all rows of the team.  Teams walk the rows with a fixed stride;
// the next row's pieces are loaded before the current row is reduced, which keeps memory busy across
// the reductions.  All arithmetic is fp32; the one rounding to bf16 is the output's.
// Bound: memory (forward 4 bytes, backward 6, with a residual gradient 8 bytes an element).  32768 x 4096: forward 90 us
// (79 at the copy rate), backward with a residual gradient 158 (158); 1237 x 2560 backward 11.5 (3.7: two launches and the
// latency of a few rows a team); one row of 4096 forward 2.4.
#include <atomic>

#include "actfn.cuh"
#include "f32x2.cuh"
#include "ops.h"
#include "ptx.cuh"

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

__device__ __forceinline__ void unpack8(const uint4& w, uint64_t (&v)[4]) {
  v[0] = f2(bf16lo(w.x), bf16hi(w.x));
  v[1] = f2(bf16lo(w.y), bf16hi(w.y));
  v[2] = f2(bf16lo(w.z), bf16hi(w.z));
  v[3] = f2(bf16lo(w.w), bf16hi(w.w));
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
// registers), y = (x - mean) rstd gamma + beta.  Where the squares leave fp32's range, of the row times 2^-80.
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
  auto gamma_at = [&](int i) {
    const int v = t + i * tpr;
    return v < nv ? reinterpret_cast<const uint4*>(a.gamma)[v] : make_uint4(0u, 0u, 0u, 0u);
  };
  auto beta_at = [&](int i) {
    const int v = t + i * tpr;
    return v < nv && a.beta ? reinterpret_cast<const uint4*>(a.beta)[v] : make_uint4(0u, 0u, 0u, 0u);
  };
  load_row<NPT>(w, a.X + r * a.ld_x, t, tpr, nv);
#pragma unroll
  for (int i = 0; i < NPT; ++i) {
    ga[i] = gamma_at(i);
    be[i] = beta_at(i);
  }
  for (; r < a.rows; r += stride) {
    uint4 next[NPT];
    const bool more = r + stride < a.rows;
    if (more) load_row<NPT>(next, a.X + (r + stride) * a.ld_x, t, tpr, nv);
    // mean and variance of the row times c
    float c = 1.0f, mean, var;
    {
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < NPT; ++i) {
        float x[8];
        unpack8(w[i], x);  // pieces past the row are zero
        s += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
      }
      mean = team_sum(s, 0.0f, red, flip, warps, team).x * inv_h;
      float q = 0.0f;
#pragma unroll
      for (int i = 0; i < NPT; ++i) {
        if (t + i * tpr >= nv) continue;
        float x[8];
        unpack8(w[i], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) q = fmaf(x[e] - mean, x[e] - mean, q);
      }
      var = team_sum(q, 0.0f, red, flip, warps, team).x * inv_h;
    }
    // Two kinds of rows are measured again (the same in the whole team), read once more: those whose squares or sums leave
    // fp32's range (or with an infinity or NaN), in a smaller scale; and those whose values are all alike, or all but one
    // (of 16384 values, one of them a bf16 step apart, the variance is 2^-30 of the mean's square), because there the error
    // of the mean, a few units of its last place, counts against the spread.  The centred values' mean takes it away
    // (all of it where they are alike).
    if (!(var < INFINITY) || var < mean * mean * 0x1p-28f) {
      c = var < INFINITY ? 1.0f : 0x1p-80f;
      mean = 0.0f;
      const uint4* again = reinterpret_cast<const uint4*>(a.X + r * a.ld_x);
#pragma unroll 1
      for (int k = 0; k < 3; ++k) {  // the mean, its correction, the variance
        float s = 0.0f;
#pragma unroll 1
        for (int v = t; v < nv; v += tpr) {
          float x[8];
          unpack8(again[v], x);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float z = fmaf(x[e], c, -mean);
            s = k == 2 ? fmaf(z, z, s) : s + z;
          }
        }
        s = team_sum(s, 0.0f, red, flip, warps, team).x * inv_h;
        if (k == 2)
          var = s;
        else
          mean += s;
      }
    }
    // (the smaller scale leaves nothing of eps: a variance of zero there is a row of one value)
    const bool alike = var == 0.0f && c != 1.0f;
    const float rstd = alike ? 0.0f : 1.0f / sqrtf(var + a.eps * c * c);
    if (t == 0) {
      if (a.mean) a.mean[r] = mean / c;
      if (a.rstd) a.rstd[r] = alike ? 1.0f / sqrtf(a.eps) : rstd * c;
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

// ---- forward of many rows: each team of `wpr` warps streams rows through its own `depth` buffers in shared memory
// with bulk copies, so that memory never waits for a reduction and no team for another.  The row is
// normalised in place and stored from there; a buffer is refilled one row after its store was issued.
// Same arithmetic as above up to the order of the sums.  32768 x 4096: 135 us above, 90 us here (0.88 of the copy
// bandwidth; the same copies without arithmetic take 86 us).
__device__ int g_norm_err;

__device__ __forceinline__ void bulk_copy_row(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void bulk_load_row(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  mbar_arrive_expect_tx(bar, bytes);
  bulk_copy_row(dst, src, bytes, bar);
}
__device__ __forceinline__ void bulk_store_row(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)), "r"(src),
               "r"(bytes)
               : "memory");
}

// After a wait that ran out: copies that other waits were for land before the block leaves.
__device__ __forceinline__ void land_copies() {
  const uint64_t t0 = global_timer_ns();
  while (global_timer_ns() - t0 < 100000ull) {
  }
}

constexpr int kStreamMaxWarps = 16, kStreamMaxDepth = 3;
constexpr int kStreamCtrl = 1024;

__global__ void __launch_bounds__(32 * kStreamMaxWarps) ln_fwd_stream_kernel(const LnFwdArgs a, const int depth, const int wpr) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, teams = (blockDim.x >> 5) / wpr;
  const int team = warp / wpr, wt = warp - team * wpr, tt = wt * 32 + lane, width = wpr * 32;
  const uint32_t row_bytes = static_cast<uint32_t>(a.h) * 2u, pitch = (row_bytes + 127u) & ~127u;
  const uint32_t bar0 = smem_u32(smem) + static_cast<uint32_t>(team * kStreamMaxDepth) * 8u;
  float* joint = reinterpret_cast<float*>(smem + 512);  // a team's warps: mean and sum of squares each
  // gamma and beta in shared memory: beside buffers of this size L1 is too small to hold them (101 -> 90 us)
  const uint32_t sg = smem_u32(smem) + kStreamCtrl, sb = sg + pitch;
  const uint32_t buf0 = sg + (2u + static_cast<uint32_t>(team * depth)) * pitch;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kStreamCtrl - 4);
  if (tt == 0) {
    for (int d = 0; d < depth; ++d) mbar_init(bar0 + 8u * d, 1);
    if (team == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  pdl_launch();
  pdl_wait();
  const int nv = static_cast<int>(a.h >> 3);
  for (int v = threadIdx.x; v < nv; v += blockDim.x) {
    const uint4 g = reinterpret_cast<const uint4*>(a.gamma)[v];
    const uint4 b = a.beta ? reinterpret_cast<const uint4*>(a.beta)[v] : make_uint4(0u, 0u, 0u, 0u);
    st_shared_v4(sg + 16u * v, g.x, g.y, g.z, g.w);
    st_shared_v4(sb + 16u * v, b.x, b.y, b.z, b.w);
  }
  __syncthreads();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * teams, r0 = static_cast<int64_t>(blockIdx.x) * teams + team;
  if (tt == 0)
    for (int d = 0; d < depth; ++d)
      if (r0 + d * stride < a.rows) bulk_load_row(buf0 + d * pitch, a.X + (r0 + d * stride) * a.ld_x, row_bytes, bar0 + 8u * d);
  auto team_sync = [&] {
    if (wpr > 1)
      asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(width) : "memory");
    else
      __syncwarp();
  };
  auto pieces = [&](int thread) { return static_cast<float>(thread < nv ? (nv - 1 - thread) / width + 1 : 0); };
  // the values (in eights) that each warp of the team holds
  auto held = [&](int w) {
    const int full = nv / width, rest = nv - full * width - w * 32;
    return static_cast<float>(full * 32 + (rest < 0 ? 0 : rest > 32 ? 32 : rest));
  };
  const float inv_h = 1.0f / static_cast<float>(a.h);
  int d = 0;
  uint32_t phase = 0;
  for (int64_t r = r0; r < a.rows; r += stride) {
    const uint32_t buf = buf0 + static_cast<uint32_t>(d) * pitch;
    // (a wait that runs out raises the abort flag; the row is then not stored)
    bool ok = mbar_wait(bar0 + 8u * d, phase, abort_flag, &g_norm_err, 0x250);
    // mean and variance of the row times c in one pass: each thread's sums are taken relative to the mean of its
    // first eight values (so that their squares do not cancel), then joined pairwise in the warp and in warp order
    auto stats = [&](float c, float& mean, float& var) {
      float n = pieces(tt), m2 = 0.0f;
      mean = 0.0f;
      if (tt < nv) {
        uint64_t x[4];
        unpack8(ld_shared_v4(buf + 16u * tt), x);
        const uint64_t c2 = f2(c, c), c8 = f2(c * 0.125f, c * 0.125f);  // (an eighth of each: their sum may leave the range)
        float lo, hi;
        f2_split(add_f2(add_f2(mul_f2(x[0], c8), mul_f2(x[1], c8)), add_f2(mul_f2(x[2], c8), mul_f2(x[3], c8))), lo, hi);
        const float shift = lo + hi;
        const uint64_t neg = f2(-shift, -shift);
        uint64_t s[2] = {0, 0}, q[2] = {0, 0};
#pragma unroll 4
        for (int v = tt; v < nv; v += width) {
          unpack8(ld_shared_v4(buf + 16u * v), x);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint64_t d2 = fma_f2(x[e], c2, neg);
            s[e & 1] = add_f2(s[e & 1], d2);
            q[e & 1] = fma_f2(d2, d2, q[e & 1]);
          }
        }
        f2_split(add_f2(s[0], s[1]), lo, hi);
        const float off = (lo + hi) / (8.0f * n);
        mean = shift + off;
        f2_split(add_f2(q[0], q[1]), lo, hi);
        m2 = (lo + hi) - off * off * (8.0f * n);
      }
      // (n, mean, m2) and (nb, mb, qb) together; n counts eights
      auto join = [](float& n, float& mean, float& m2, float nb, float mb, float qb) {
        const float both = n + nb, w = both > 0.0f ? nb / both : 0.0f, diff = mb - mean;
        m2 = m2 + qb + diff * diff * (8.0f * n * w);
        mean = mean + diff * w;
        n = both;
      };
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float nb = __shfl_xor_sync(0xFFFFFFFFu, n, o), mb = __shfl_xor_sync(0xFFFFFFFFu, mean, o);
        join(n, mean, m2, nb, mb, __shfl_xor_sync(0xFFFFFFFFu, m2, o));
      }
      if (wpr > 1) {
        if (lane == 0) {
          joint[2 * warp] = mean;
          joint[2 * warp + 1] = m2;
        }
        team_sync();
        const float* j = joint + 2 * team * wpr;
        n = held(0);
        mean = j[0];
        m2 = j[1];
        for (int w = 1; w < wpr; ++w) join(n, mean, m2, held(w), j[2 * w], j[2 * w + 1]);
      } else {  // lanes may differ in the last bit
        mean = __shfl_sync(0xFFFFFFFFu, mean, 0);
        m2 = __shfl_sync(0xFFFFFFFFu, m2, 0);
      }
      // infinite or NaN: squares beyond fp32 (also as inf - inf above), or an infinity or NaN in the row
      var = fabsf(m2) < INFINITY ? fmaxf(m2, 0.0f) * inv_h : NAN;
    };
    float c = 1.0f, mean, var;
    stats(1.0f, mean, var);
    if (!(var < INFINITY) || !(fabsf(mean) < INFINITY)) {  // as in ln_fwd_kernel; the same in the whole team
      c = 0x1p-80f;
      team_sync();  // the first sums are read
      stats(c, mean, var);
    }
    const float rstd = 1.0f / sqrtf(var + a.eps * c * c);
    if (tt == 0) {
      if (a.mean) a.mean[r] = mean / c;
      if (a.rstd) a.rstd[r] = rstd * c;
    }
    const uint64_t c2 = f2(c, c), neg = f2(-mean, -mean), r2 = f2(rstd, rstd);
#pragma unroll 4
    for (int v = tt; v < nv; v += width) {
      uint64_t x[4], g[4], b[4];
      unpack8(ld_shared_v4(buf + 16u * v), x);
      unpack8(ld_shared_v4(sg + 16u * v), g);
      unpack8(ld_shared_v4(sb + 16u * v), b);
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float lo, hi;
        f2_split(fma_f2(mul_f2(fma_f2(x[e], c2, neg), r2), g[e], b[e]), lo, hi);
        y[e] = pack_bf16x2(lo, hi);
      }
      st_shared_v4(buf + 16u * v, y[0], y[1], y[2], y[3]);
    }
    fence_proxy_async_smem();
    team_sync();  // the row is written, and the joint sums are read
    if (tt == 0 && ok && !*abort_flag) {
      bulk_store_row(a.Y + r * a.ld_y, buf, row_bytes);
      bulk_commit_group();
      // the previous row's buffer: its store has read it once at most this row's is pending
      const int64_t next = r + (depth - 1) * stride;
      if (r != r0 && next < a.rows) {
        bulk_wait_group_read<1>();
        const int pd = d == 0 ? depth - 1 : d - 1;
        bulk_load_row(buf0 + static_cast<uint32_t>(pd) * pitch, a.X + next * a.ld_x, row_bytes, bar0 + 8u * pd);
      }
    }
    if (++d == depth) {
      d = 0;
      phase ^= 1u;
    }
  }
  if (tt == 0) bulk_wait_group_all();
  if (*abort_flag) land_copies();
  __syncwarp();
}

// With u = gy gamma and n = (x - mean) rstd:  gx = rstd (u - mean(u) - n mean(u n)) (+ gres);
// the columns' sums of gy n and gy over the block's rows go to row blockIdx.x of `part` (2 h floats).
template <int NPT, bool PREFETCH>
__global__ void __launch_bounds__(kTeamThreads) ln_bwd_kernel(const LnBwdArgs a, float* part,
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

// ---- backward of many rows: as the forward's, teams of `wpr` warps stream gY, X and the residual's gradient (`ops` rows
// a buffer set) through `depth` buffer sets of their own; a thread keeps its columns' sums (NPT pieces of eight) in
// registers over all rows of its team.  Same arithmetic as ln_bwd_kernel up to the order of the sums.  Sixteen warps of
// up to 128 registers: as few a row as four pieces a thread allow, because a row's reduction costs more than its
// arithmetic (26715 x 4096: 115 us; with 24 warps of at most two pieces 162; with 8 of at most eight 114, but 59 instead
// of 36 at 1024 columns).  32768 x 4096 with a residual's gradient 158 us, which is the copy rate; teams 183.
template <int NPT>
__global__ void __launch_bounds__(32 * kStreamMaxWarps)
    ln_bwd_stream_kernel(const LnBwdArgs a, float* part, const int depth, const int wpr) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, teams = (blockDim.x >> 5) / wpr;
  const int team = warp / wpr, wt = warp - team * wpr, tt = wt * 32 + lane, width = wpr * 32;
  const uint32_t row_bytes = static_cast<uint32_t>(a.h) * 2u, pitch = (row_bytes + 127u) & ~127u;
  const uint32_t ops = a.gres ? 3u : 2u, set = ops * pitch;
  const uint32_t bar0 = smem_u32(smem) + static_cast<uint32_t>(team * kStreamMaxDepth) * 8u;
  float2* joint = reinterpret_cast<float2*>(smem + 512);  // a warp's sums of u and u n
  const uint32_t sg = smem_u32(smem) + kStreamCtrl, ring = sg + pitch;
  const uint32_t buf0 = ring + static_cast<uint32_t>(team * depth) * set;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kStreamCtrl - 4);
  if (tt == 0) {
    for (int d = 0; d < depth; ++d) mbar_init(bar0 + 8u * d, 1);
    if (team == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  pdl_launch();
  pdl_wait();
  const int nv = static_cast<int>(a.h >> 3);
  for (int v = threadIdx.x; v < nv; v += blockDim.x) {
    const uint4 g = reinterpret_cast<const uint4*>(a.gamma)[v];
    st_shared_v4(sg + 16u * v, g.x, g.y, g.z, g.w);
  }
  __syncthreads();
  const int64_t stride = static_cast<int64_t>(gridDim.x) * teams, r0 = static_cast<int64_t>(blockIdx.x) * teams + team;
  auto load = [&](int64_t r, int d) {
    const uint32_t buf = buf0 + static_cast<uint32_t>(d) * set, bar = bar0 + 8u * d;
    mbar_arrive_expect_tx(bar, ops * row_bytes);
    bulk_copy_row(buf, a.gY + r * a.ld_gy, row_bytes, bar);
    bulk_copy_row(buf + pitch, a.X + r * a.ld_x, row_bytes, bar);
    if (a.gres) bulk_copy_row(buf + 2 * pitch, a.gres + r * a.ld_gres, row_bytes, bar);
  };
  if (tt == 0)
    for (int d = 0; d < depth; ++d)
      if (r0 + d * stride < a.rows) load(r0 + d * stride, d);
  auto team_sync = [&] {
    if (wpr > 1)
      asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(width) : "memory");
    else
      __syncwarp();
  };
  const float inv_h = 1.0f / static_cast<float>(a.h);
  uint64_t ag[NPT][4], ab[NPT][4];
#pragma unroll
  for (int i = 0; i < NPT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) ag[i][e] = ab[i][e] = 0;
  float mean = 0.0f, rstd = 0.0f;
  if (r0 < a.rows) {
    mean = a.mean[r0];
    rstd = a.rstd[r0];
  }
  int d = 0;
  uint32_t phase = 0;
  for (int64_t r = r0; r < a.rows; r += stride) {
    const uint32_t buf = buf0 + static_cast<uint32_t>(d) * set;
    const bool more = r + stride < a.rows;
    const float nmean = more ? a.mean[r + stride] : 0.0f, nrstd = more ? a.rstd[r + stride] : 0.0f;
    const uint64_t neg = f2(-mean, -mean), scale = f2(rstd, rstd);
    // (a wait that runs out raises the abort flag; the rows after it are neither loaded nor stored)
    const bool ok = mbar_wait(bar0 + 8u * d, phase, abort_flag, &g_norm_err, 0x251);
    uint64_t su = 0, sun = 0;
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
      const int v = tt + i * width;
      if (v >= nv) continue;
      uint64_t g[4], x[4], m[4];
      unpack8(ld_shared_v4(buf + 16u * v), g);
      unpack8(ld_shared_v4(buf + pitch + 16u * v), x);
      unpack8(ld_shared_v4(sg + 16u * v), m);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t n = mul_f2(add_f2(x[e], neg), scale), u = mul_f2(g[e], m[e]);
        su = add_f2(su, u);
        sun = fma_f2(u, n, sun);
        ag[i][e] = fma_f2(g[e], n, ag[i][e]);
        ab[i][e] = add_f2(ab[i][e], g[e]);
      }
    }
    float2 s;
    {
      float lo, hi;
      f2_split(su, lo, hi);
      s.x = lo + hi;
      f2_split(sun, lo, hi);
      s.y = lo + hi;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s.x += __shfl_xor_sync(0xFFFFFFFFu, s.x, o);
      s.y += __shfl_xor_sync(0xFFFFFFFFu, s.y, o);
    }
    if (wpr > 1) {
      if (lane == 0) joint[warp] = s;
      team_sync();
      s = joint[team * wpr];
      for (int w = 1; w < wpr; ++w) {
        const float2 o = joint[team * wpr + w];
        s.x += o.x;
        s.y += o.y;
      }
    }
    const float mu = s.x * inv_h, mun = s.y * inv_h;
    const uint64_t nmu = f2(-mu, -mu), nmun = f2(-mun, -mun);
    uint4* out = reinterpret_cast<uint4*>(a.gX + r * a.ld_gx);
#pragma unroll
    for (int i = 0; i < NPT; ++i) {
      const int v = tt + i * width;
      if (v >= nv) continue;
      uint64_t g[4], x[4], m[4], z[4] = {0, 0, 0, 0};
      unpack8(ld_shared_v4(buf + 16u * v), g);
      unpack8(ld_shared_v4(buf + pitch + 16u * v), x);
      unpack8(ld_shared_v4(sg + 16u * v), m);
      if (a.gres) unpack8(ld_shared_v4(buf + 2 * pitch + 16u * v), z);
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t n = mul_f2(add_f2(x[e], neg), scale), u = mul_f2(g[e], m[e]);
        float lo, hi;
        f2_split(fma_f2(scale, fma_f2(n, nmun, add_f2(u, nmu)), z[e]), lo, hi);
        y[e] = pack_bf16x2(lo, hi);
      }
      if (ok) out[v] = make_uint4(y[0], y[1], y[2], y[3]);
    }
    team_sync();  // the buffers and the joint sums are read
    if (tt == 0 && ok && !*abort_flag && r + depth * stride < a.rows) load(r + depth * stride, d);
    mean = nmean;
    rstd = nrstd;
    if (++d == depth) {
      d = 0;
      phase ^= 1u;
    }
  }
  if (*abort_flag) land_copies();
  // the teams' sums in team order
  float* out = part + static_cast<int64_t>(blockIdx.x) * 2 * a.h;
  float* cols = teams == 1 ? out : reinterpret_cast<float*>(smem + kStreamCtrl + pitch);
  __syncthreads();  // every team is done with the ring
#pragma unroll
  for (int i = 0; i < NPT; ++i) {
    const int c = (tt + i * width) * 8;
    if (c >= a.h) continue;
    float* to = cols + static_cast<int64_t>(team) * 2 * a.h + c;
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      float4 s;
      f2_split(ag[i][e], s.x, s.y);
      f2_split(ag[i][e + 1], s.z, s.w);
      *reinterpret_cast<float4*>(to + 2 * e) = s;
      f2_split(ab[i][e], s.x, s.y);
      f2_split(ab[i][e + 1], s.z, s.w);
      *reinterpret_cast<float4*>(to + a.h + 2 * e) = s;
    }
  }
  if (teams == 1) return;
  __syncthreads();
  for (int64_t c = threadIdx.x * 4; c < 2 * a.h; c += blockDim.x * 4) {
    float4 s = *reinterpret_cast<const float4*>(cols + c);
    for (int k = 1; k < teams; ++k) {
      const float4 o = *reinterpret_cast<const float4*>(cols + k * 2 * a.h + c);
      s.x += o.x; s.y += o.y; s.z += o.z; s.w += o.w;
    }
    *reinterpret_cast<float4*>(out + c) = s;
  }
}

// Column sums of `parts` rows of 2 h floats, in a fixed order: 32 groups of rows per block, then the
// groups in order.  Columns 0 .. h-1 go to ggamma, the others to gbeta (nullable).
__global__ void __launch_bounds__(1024) ln_cols_kernel(const float* part, int parts, int64_t h,
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

constexpr int kMaxSmem = 232448;  // a CTA's
// Forward: a row of up to 1024 columns is one warp's where there are rows to fill the GPU so (no barrier; 26715 rows of
// 584: 18.1 us, with three warps a row 29.4, streamed 24.8; of 1024: 24.9, 32.6, 27.3), but several warps' where there
// are few (64 rows of 904: 2.0 us, one warp a row 2.4).  Wider rows are streamed from 2.2 M values on: at 4096 columns
// the two cross at 650 rows (11.0 and 6.5 us at 1216), at 1200 at 1800 (1000 rows: 3.3, streamed 4.4; 6648: 15.4 and 10.3).
constexpr int64_t kNarrowMinRows = 512, kStreamMinH = 1032, kStreamMinValues = 2200000;
// Backward: streamed from 1 M values on.  Teams and streamed, us, without a residual's gradient: 26715 rows of 584 41 and
// 27, of 1576 82 and 60, of 2056 116 and 70, of 4096 127 and 115; 1000 rows of 1576 8.6 and 8.2, of 4096 12.5 and 12.4;
// 8 rows of 1576 5.0 and 6.8.
constexpr int64_t kStreamBwdMinValues = 1000000;
int pieces_per_thread(int64_t h) { return h <= 2048 ? 1 : (h <= 8192 ? 2 : 4); }
int team_threads(int64_t h, int npt) { return static_cast<int>(((h / 8 + npt - 1) / npt + 31) / 32 * 32); }

}  // namespace

namespace {
bool ln_bwd_streams(int64_t rows, int64_t h) { return rows * h >= kStreamBwdMinValues; }
// warps a row: at most four pieces of eight columns a thread
int stream_bwd_warps(int64_t h) { return static_cast<int>((h + 1023) / 1024); }
}  // namespace

int ln_bwd_blocks(int64_t rows, int64_t h, int sms) {
  if (ln_bwd_streams(rows, h)) {
    const int teams = kStreamMaxWarps / stream_bwd_warps(h);
    const int64_t need = (rows + teams - 1) / teams;
    return static_cast<int>(need < sms ? need : sms);
  }
  const int tpr = team_threads(h, pieces_per_thread(h)), teams = tpr >= 256 ? 1 : 256 / tpr;
  const int64_t need = (rows + 4 * teams - 1) / (4 * teams), most = 2 * int64_t(sms);
  return static_cast<int>(need < most ? need : most);
}

namespace {
cudaError_t launch_ln_fwd_stream(const LnFwdArgs& a, int sms, cudaStream_t st) {
  static std::atomic<bool> ready_of[kMaxDevices];  // the shared-memory opt-in, per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!ready_of[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(ln_fwd_stream_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    ready_of[dev].store(true, std::memory_order_release);
  }
  // as many teams as rows fit beside gamma and beta, sixteen warps among them
  const int64_t pitch = (a.h * 2 + 127) / 128 * 128;
  const int depth = pitch > 16384 ? 2 : 3;
  const int64_t fit = (kMaxSmem - kStreamCtrl - 2 * pitch) / (pitch * depth);
  const int teams = static_cast<int>(fit < kStreamMaxWarps ? fit : kStreamMaxWarps);
  const int wpr = teams > 8 ? 1 : teams > 4 ? 2 : teams > 2 ? 4 : 8;
  return launch_pdl(ln_fwd_stream_kernel, dim3(static_cast<unsigned>(sms)), dim3(static_cast<unsigned>(32 * wpr * teams)),
                    size_t(kStreamCtrl + pitch * (2 + depth * teams)), 1, st, a, depth, wpr);
}
}  // namespace

cudaError_t launch_ln_fwd(const LnFwdArgs& a, int sms, cudaStream_t st) {
  if (a.rows == 0) return cudaSuccess;
  if (a.h >= kStreamMinH && a.rows * a.h >= kStreamMinValues) return launch_ln_fwd_stream(a, sms, st);
  const int npt = a.rows < kNarrowMinRows ? pieces_per_thread(a.h) : a.h <= 1024 ? static_cast<int>((a.h + 255) / 256)
                                                                  : a.h <= 2048 ? 4 : pieces_per_thread(a.h);
  const int tpr = team_threads(a.h, npt), teams = tpr >= 256 ? 1 : 256 / tpr;
  const int64_t need = (a.rows + teams - 1) / teams, most = int64_t(sms) * (2048 / (teams * tpr));
  const dim3 grid(static_cast<unsigned>(need < most ? need : most)), block(static_cast<unsigned>(teams * tpr));
  const auto fn = npt == 1 ? ln_fwd_kernel<1> : npt == 2 ? ln_fwd_kernel<2> : npt == 3 ? ln_fwd_kernel<3> : ln_fwd_kernel<4>;
  return launch_pdl(fn, grid, block, 0, 1, st, a, tpr);
}

namespace {
cudaError_t launch_ln_bwd_stream(const LnBwdArgs& a, float* part, int grid, cudaStream_t st) {
  const int wpr = stream_bwd_warps(a.h), teams = kStreamMaxWarps / wpr;
  const int npt = static_cast<int>((a.h / 8 + 32 * wpr - 1) / (32 * wpr));
  const auto fn = npt == 1 ? ln_bwd_stream_kernel<1> : npt == 2 ? ln_bwd_stream_kernel<2> : npt == 3 ? ln_bwd_stream_kernel<3>
                                                                                                 : ln_bwd_stream_kernel<4>;
  static std::atomic<bool> ready_of[4][kMaxDevices];  // the shared-memory opt-in, per instance and device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!ready_of[npt - 1][dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    ready_of[npt - 1][dev].store(true, std::memory_order_release);
  }
  // two buffer sets always fit (at most 16384 columns a set), and hold the teams' sums at the end
  const int64_t pitch = (a.h * 2 + 127) / 128 * 128, set = pitch * (a.gres ? 3 : 2) * teams;
  const int64_t fit = (kMaxSmem - kStreamCtrl - pitch) / set;
  const int depth = static_cast<int>(fit < kStreamMaxDepth ? fit : kStreamMaxDepth);
  return launch_pdl(fn, dim3(static_cast<unsigned>(grid)), dim3(static_cast<unsigned>(32 * wpr * teams)), size_t(kStreamCtrl + pitch + depth * set), 1, st, a,
                    part, depth, wpr);
}
}  // namespace

cudaError_t launch_ln_bwd(const LnBwdArgs& a, float* part, int sms, cudaStream_t st) {
  const int grid = ln_bwd_blocks(a.rows, a.h, sms);
  if (grid == 0) return cudaSuccess;
  if (ln_bwd_streams(a.rows, a.h)) return launch_ln_bwd_stream(a, part, grid, st);
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

cudaError_t take_norm_error(int* code) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_norm_err, sizeof(int));
  if (e != cudaSuccess) return e;
  *code = v;
  if (v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_norm_err, &zero, sizeof(int));
  }
  return e;
}

}  // namespace dm
