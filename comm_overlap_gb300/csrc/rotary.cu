// rotary.cu -- what stands between the fused projection and the attention: the norm of each query and key head with the
// rotation by position (forward, backward), and the 8-bit cache of keys and values (written in the same pass, read back).
//
// A head's 128 values are held by 8 lanes of a warp, two 16-byte pieces each, chosen so that a rotated pair always lies in one
// lane: with rot = 16 m rotated values, lane j < m holds pieces j and j + m (half layout: value i pairs with i + rot / 2, which
// is m pieces further; interleaved: 2 i with 2 i + 1, in one piece), the lanes from m on two neighbouring pieces of the rest.
// A warp takes four heads at a time, all of one token, whose cosines and sines it computes once.
//
// Angles: a position turns pair i by position x frequency.  The frequency is kept as a 64-bit fraction of a turn, so the
// product's low 64 bits are the angle's fraction of a turn without any rounding by the position's size; its upper 32 bits go to
// sincospif.
//
// Bound: memory.  Forward 4 bytes a value, backward 6 (4 without norm), cache 3.
#include <atomic>

#include "actfn.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace dm {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kHeadsAbreast = 4;  // heads of a warp's step

__device__ int g_rotary_err;

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  v[0] = bf16lo(w.x); v[1] = bf16hi(w.x); v[2] = bf16lo(w.y); v[3] = bf16hi(w.y);
  v[4] = bf16lo(w.z); v[5] = bf16hi(w.z); v[6] = bf16lo(w.w); v[7] = bf16hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// Frequency (radians a position) as a fraction of a turn, in units of 2^-64 turns.
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
  double t = f * 0.15915494309189533577;
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);
}

// The lanes' places in a head: pieces ca and cb, and whether they are rotated.
struct Place {
  int slot, j, ca, cb;
  bool turns;
};
__device__ __forceinline__ Place place_of(int lane, int rot) {
  Place p;
  const int m = rot >> 4;
  p.slot = lane >> 3;
  p.j = lane & 7;
  p.turns = p.j < m;
  p.ca = p.turns ? p.j : 2 * p.j;
  p.cb = p.turns ? p.j + m : 2 * p.j + 1;
  return p;
}

// Cosines and sines of a token's angles, times the amplitude: computed by the warp's lanes, two pairs each, and read back from
// shared memory (64 float2 a warp) in the order of the lane's own pairs: half layout 8 j + e for (a[e], b[e]); interleaved
// 4 ca + i for (a[2 i], a[2 i + 1]) and 4 cb + i for b's.
template <bool HALF>
__device__ __forceinline__ void token_angles(float2* mine, const unsigned long long* turns, int position, int rot, float amplitude,
                                             int lane, const Place& p, float (&c)[8], float (&s)[8]) {
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    if (i < (rot >> 1)) {
      const unsigned long long at = turns[i] * static_cast<unsigned long long>(static_cast<long long>(position));
      float sn, cs;
      sincospif(static_cast<float>(static_cast<int>(at >> 32)) * 0x1p-31f, &sn, &cs);
      mine[i] = make_float2(cs * amplitude, sn * amplitude);
    }
  }
  __syncwarp();
  if (p.turns) {
    const int first = HALF ? 8 * p.j : 4 * p.ca, second = HALF ? 8 * p.j + 4 : 4 * p.cb;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const float4 x = *reinterpret_cast<const float4*>(mine + first + i), y = *reinterpret_cast<const float4*>(mine + second + i);
      c[i] = x.x; s[i] = x.y; c[i + 1] = x.z; s[i + 1] = x.w;
      c[i + 4] = y.x; s[i + 4] = y.y; c[i + 5] = y.z; s[i + 5] = y.w;
    }
  }
}

template <bool HALF>
__device__ __forceinline__ void rotate(float (&a)[8], float (&b)[8], const float (&c)[8], const float (&s)[8], float sign) {
  if (HALF) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = a[e], y = b[e], sn = s[e] * sign;
      a[e] = fmaf(x, c[e], -y * sn);
      b[e] = fmaf(x, sn, y * c[e]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = a[2 * i], y = a[2 * i + 1], sn = s[i] * sign;
      a[2 * i] = fmaf(x, c[i], -y * sn);
      a[2 * i + 1] = fmaf(x, sn, y * c[i]);
      const float z = b[2 * i], w = b[2 * i + 1], sm = s[i + 4] * sign;
      b[2 * i] = fmaf(z, c[i + 4], -w * sm);
      b[2 * i + 1] = fmaf(z, sm, w * c[i + 4]);
    }
  }
}

__device__ __forceinline__ float head_sum(float v) {  // over the 8 lanes of a head, the same bits in each
  v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
  v += __shfl_xor_sync(0xFFFFFFFFu, v, 2);
  return v + __shfl_xor_sync(0xFFFFFFFFu, v, 4);
}
__device__ __forceinline__ float head_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
  v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
  return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
}

__device__ __forceinline__ float squares(const float (&a)[8], const float (&b)[8]) {
  float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    s0 = fmaf(a[e], a[e], s0);
    s1 = fmaf(b[e], b[e], s1);
  }
  return s0 + s1;
}

constexpr float kInvD = 1.0f / 128.0f;
// Heads whose squares leave fp32's range are measured times this.
constexpr float kSmaller = 0x1p-80f;

// x / sqrt(mean(x^2) + eps) times the weight (bf16 pieces wa, wb).
__device__ __forceinline__ void normalise(float (&a)[8], float (&b)[8], const uint4& wa, const uint4& wb, float eps) {
  float ss = head_sum(squares(a, b)), c = 1.0f;
  if (__any_sync(0xFFFFFFFFu, !(ss < INFINITY))) {
    c = ss < INFINITY ? 1.0f : kSmaller;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[e] *= c;
      b[e] *= c;
    }
    ss = head_sum(squares(a, b));
  }
  const float rstd = rsqrtf(fmaf(ss, kInvD, eps * c * c));
  float w[8];
  unpack8(wa, w);
#pragma unroll
  for (int e = 0; e < 8; ++e) a[e] *= rstd * w[e];
  unpack8(wb, w);
#pragma unroll
  for (int e = 0; e < 8; ++e) b[e] *= rstd * w[e];
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }

// E4M3 codes of a head: the least e with amax <= 448 x 2^e (1.75 x 2^8), in [-kCacheExpMax, kCacheExpMax] (0 for a head of
// zeros), then x 2^-e, which is exact, rounded once.  An infinity becomes NaN, and counts no more than one for e.
__device__ __forceinline__ int quantise(float (&a)[8], float (&b)[8], uint2& qa, uint2& qb) {
  float amax = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(fabsf(a[e]), fabsf(b[e])));
  amax = head_max(amax);
  if (__any_sync(0xFFFFFFFFu, !(amax < INFINITY))) {
    amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[e] = fabsf(a[e]) < INFINITY ? a[e] : NAN;
      b[e] = fabsf(b[e]) < INFINITY ? b[e] : NAN;
      amax = fmaxf(amax, fmaxf(fabsf(a[e]), fabsf(b[e])));  // (NaN is passed over)
    }
    amax = head_max(amax);
  }
  const uint32_t bits = __float_as_uint(amax);
  int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u);
  e = amax > 0.0f ? min(max(e, -kCacheExpMax), kCacheExpMax) : 0;
  const float f = power_of_two(-e);
  qa = make_uint2(e4m3x4(a[0] * f, a[1] * f, a[2] * f, a[3] * f), e4m3x4(a[4] * f, a[5] * f, a[6] * f, a[7] * f));
  qb = make_uint2(e4m3x4(b[0] * f, b[1] * f, b[2] * f, b[3] * f), e4m3x4(b[4] * f, b[5] * f, b[6] * f, b[7] * f));
  return e;
}

// ---- forward: a unit is a token's part of its groups of four heads (queries, then keys, then, into the cache, values)
template <bool NORM, bool HALF, bool CACHE>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a, const int split) {
  __shared__ unsigned long long turns[64];
  __shared__ float2 angles[kWarps][64];
  pdl_launch();
  pdl_wait();
  if (static_cast<int>(threadIdx.x) < (a.rot >> 1)) turns[threadIdx.x] = turn_fraction(a.frequencies[threadIdx.x]);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Place p = place_of(lane, a.rot);
  const int gq = (a.hq + kHeadsAbreast - 1) / kHeadsAbreast, gk = (a.hkv + kHeadsAbreast - 1) / kHeadsAbreast;
  const int groups = gq + gk + (CACHE ? gk : 0);
  uint4 wqa = {}, wqb = {}, wka = {}, wkb = {};
  if (NORM) {
    wqa = reinterpret_cast<const uint4*>(a.wq)[p.ca];
    wqb = reinterpret_cast<const uint4*>(a.wq)[p.cb];
    if (a.wk) {
      wka = reinterpret_cast<const uint4*>(a.wk)[p.ca];
      wkb = reinterpret_cast<const uint4*>(a.wk)[p.cb];
    }
  }
  const int64_t units = a.tokens * split, stride = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kWarps + warp; u < units; u += stride) {
    const int64_t token = split == 1 ? u : u / split;
    const int part = static_cast<int>(u - token * split);
    int row = 0;
    bool write = true;
    if (CACHE) {
      row = a.rows[token];
      write = row >= 0 && row < a.cache_rows;
      if (row >= a.cache_rows && lane == 0) atomicCAS(&g_rotary_err, 0, kPackedBadLengths);
    }
    // the head of this lane in a group, and its pieces in memory (null past the last head)
    auto source = [&](int group) -> const uint16_t* {
      const int which = group < gq ? 0 : group < gq + gk ? 1 : 2;
      const int head = (group - (which == 0 ? 0 : which == 1 ? gq : gq + gk)) * kHeadsAbreast + p.slot;
      if (head >= (which == 0 ? a.hq : a.hkv)) return nullptr;
      return (which == 0 ? a.Q + token * a.ld_q : which == 1 ? a.K + token * a.ld_k : a.V + token * a.ld_v) + head * 128;
    };
    auto load = [&](int group, uint4& xa, uint4& xb) {
      const uint16_t* x = group < groups ? source(group) : nullptr;
      xa = x ? __ldcs(reinterpret_cast<const uint4*>(x) + p.ca) : make_uint4(0u, 0u, 0u, 0u);
      xb = x ? __ldcs(reinterpret_cast<const uint4*>(x) + p.cb) : make_uint4(0u, 0u, 0u, 0u);
    };
    // two groups in flight, in registers of their own each (moved from one to the other they were waited for: 69 us for 16384
    // tokens of 32 + 8 heads)
    uint4 xa, xb, ya, yb;
    load(part, xa, xb);
    load(part + split, ya, yb);
    float c[8], s[8];
    if (a.rot > 0)
      token_angles<HALF>(angles[warp], turns, a.positions[token], a.rot, a.amplitude, lane, p, c, s);
    auto step = [&](int group, uint4& wa, uint4& wb) {
      float va[8], vb[8];
      unpack8(wa, va);
      unpack8(wb, vb);
      load(group + 2 * split, wa, wb);
      const bool query = group < gq, value = CACHE && group >= gq + gk;
      if (!value) {
        if (NORM) normalise(va, vb, query ? wqa : wka, query ? wqb : wkb, a.eps);
        if (p.turns) rotate<HALF>(va, vb, c, s, a.sign);
      }
      const int head = (group - (query ? 0 : value ? gq + gk : gq)) * kHeadsAbreast + p.slot;
      if (CACHE && !query) {
        uint2 qa, qb;
        const int e = quantise(va, vb, qa, qb);
        if (write && head < a.hkv) {
          uint8_t* codes = (value ? a.v8 : a.k8) + (static_cast<int64_t>(row) * a.hkv + head) * 128;
          reinterpret_cast<uint2*>(codes)[p.ca] = qa;
          reinterpret_cast<uint2*>(codes)[p.cb] = qb;
          if (p.j == 0) (value ? a.v_exp : a.k_exp)[head * a.ld_exp + row] = static_cast<uint8_t>(e + 127);
        }
      } else if (head < (query ? a.hq : a.hkv)) {
        uint16_t* y = (query ? a.Yq + token * a.ld_yq : a.Yk + token * a.ld_yk) + head * 128;
        reinterpret_cast<uint4*>(y)[p.ca] = pack8(va);
        reinterpret_cast<uint4*>(y)[p.cb] = pack8(vb);
      }
    };
    for (int group = part; group < groups; group += 2 * split) {
      step(group, xa, xb);
      if (group + split < groups) step(group + split, ya, yb);
    }
  }
}

// ---- backward with norm.  With u = amplitude R^T gy, n = x rstd: gx = rstd (u w - n mean(u w n)), gw = sum of u n over tokens
// and heads.  Each lane adds up its values' gw in registers over all its heads; a block leaves 256 sums (queries', keys').
template <bool HALF>
__global__ void __launch_bounds__(kThreads) rotary_bwd_kernel(const RotaryBwdArgs a, float* part, const int split) {
  __shared__ unsigned long long turns[64];
  __shared__ float2 angles[kWarps][64];
  __shared__ float sums[kWarps][256];
  pdl_launch();
  pdl_wait();
  if (static_cast<int>(threadIdx.x) < (a.rot >> 1)) turns[threadIdx.x] = turn_fraction(a.frequencies[threadIdx.x]);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Place p = place_of(lane, a.rot);
  const int gq = (a.hq + kHeadsAbreast - 1) / kHeadsAbreast, groups = gq + (a.hkv + kHeadsAbreast - 1) / kHeadsAbreast;
  float acc[2][16];
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[0][e] = acc[1][e] = 0.0f;
  const int64_t units = a.tokens * split, stride = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp; unit < units; unit += stride) {
    const int64_t token = split == 1 ? unit : unit / split;
    const int first = static_cast<int>(unit - token * split);
    auto load = [&](int group, uint4 (&x)[4]) {
      const bool query = group < gq;
      const int head = (group - (query ? 0 : gq)) * kHeadsAbreast + p.slot;
      if (group < groups && head < (query ? a.hq : a.hkv)) {
        const uint4* g = reinterpret_cast<const uint4*>((query ? a.gYq + token * a.ld_gyq : a.gYk + token * a.ld_gyk) + head * 128);
        const uint4* v = reinterpret_cast<const uint4*>((query ? a.Q + token * a.ld_q : a.K + token * a.ld_k) + head * 128);
        x[0] = __ldcs(g + p.ca);
        x[1] = __ldcs(g + p.cb);
        x[2] = __ldcs(v + p.ca);
        x[3] = __ldcs(v + p.cb);
      } else {
        x[0] = x[1] = x[2] = x[3] = make_uint4(0u, 0u, 0u, 0u);
      }
    };
    uint4 x0[4], x1[4];
    load(first, x0);
    load(first + split, x1);
    float c[8], s[8];
    if (a.rot > 0) token_angles<HALF>(angles[warp], turns, a.positions[token], a.rot, a.amplitude, lane, p, c, s);
    auto step = [&](int group, uint4 (&now)[4]) {
      const bool query = group < gq;
      const uint16_t* weight = query ? a.wq : a.wk;
      float ua[8], ub[8], xa[8], xb[8], wa[8], wb[8];
      unpack8(now[0], ua);
      unpack8(now[1], ub);
      unpack8(now[2], xa);
      unpack8(now[3], xb);
      load(group + 2 * split, now);
      unpack8(reinterpret_cast<const uint4*>(weight)[p.ca], wa);
      unpack8(reinterpret_cast<const uint4*>(weight)[p.cb], wb);
      if (p.turns) rotate<HALF>(ua, ub, c, s, -1.0f);
      float small = 1.0f, ss = head_sum(squares(xa, xb));
      if (__any_sync(0xFFFFFFFFu, !(ss < INFINITY))) {  // as in normalise
        small = ss < INFINITY ? 1.0f : kSmaller;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          xa[e] *= small;
          xb[e] *= small;
        }
        ss = head_sum(squares(xa, xb));
      }
      const float rstd = rsqrtf(fmaf(ss, kInvD, a.eps * small * small));
      float dot = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xa[e] *= rstd;
        xb[e] *= rstd;
        if (query) {
          acc[0][e] = fmaf(ua[e], xa[e], acc[0][e]);
          acc[0][8 + e] = fmaf(ub[e], xb[e], acc[0][8 + e]);
        } else {
          acc[1][e] = fmaf(ua[e], xa[e], acc[1][e]);
          acc[1][8 + e] = fmaf(ub[e], xb[e], acc[1][8 + e]);
        }
        ua[e] *= wa[e];
        ub[e] *= wb[e];
        dot = fmaf(ua[e], xa[e], dot);
        dot = fmaf(ub[e], xb[e], dot);
      }
      const float m = head_sum(dot) * kInvD, r = rstd * small;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ua[e] = r * fmaf(-xa[e], m, ua[e]);
        ub[e] = r * fmaf(-xb[e], m, ub[e]);
      }
      const int head = (group - (query ? 0 : gq)) * kHeadsAbreast + p.slot;
      if (head < (query ? a.hq : a.hkv)) {
        uint16_t* y = (query ? a.gQ + token * a.ld_gq : a.gK + token * a.ld_gk) + head * 128;
        reinterpret_cast<uint4*>(y)[p.ca] = pack8(ua);
        reinterpret_cast<uint4*>(y)[p.cb] = pack8(ub);
      }
    };
    for (int group = first; group < groups; group += 2 * split) {
      step(group, x0);
      if (group + split < groups) step(group + split, x1);
    }
  }
  // over the warp's four heads, then the block's warps in order
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float v = acc[k][e];
      v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
      v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
      if (p.slot == 0) sums[warp][128 * k + 8 * (e < 8 ? p.ca : p.cb) + (e & 7)] = v;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < 256; i += kThreads) {
    float v = sums[0][i];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) v += sums[w][i];
    part[static_cast<int64_t>(blockIdx.x) * 256 + i] = v;
  }
}

// The blocks' sums, added up in order by 8 rows of threads and then across them; one block for 32 columns.
__global__ void __launch_bounds__(256) rotary_sums_kernel(const RotaryBwdArgs a, const float* part, const int blocks) {
  __shared__ float rows[8][32];
  pdl_launch();
  pdl_wait();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, col = blockIdx.x * 32 + x;
  float v = 0.0f;
#pragma unroll 4
  for (int b = y; b < blocks; b += 8) v += part[static_cast<int64_t>(b) * 256 + col];
  rows[y][x] = v;
  __syncthreads();
  if (y != 0) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) v += rows[i][x];
  float* to = col < 128 ? a.gwq + col : a.gwk ? a.gwk + (col - 128) : nullptr;
  if (to) *to = a.accumulate ? *to + v : v;
}

// ---- cache, read back: a thread takes 16 codes
__device__ __forceinline__ uint32_t half2_of_e4m3x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_of_e4m3x2(uint32_t two, float f) {
  float lo, hi;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(half2_of_e4m3x2(two)));
  return pack_bf16x2(lo * f, hi * f);  // (exact)
}
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheReadArgs a) {
  pdl_launch();
  pdl_wait();
  const int per = a.hkv * 8;  // pieces of a token in one of K and V
  const int64_t pieces = a.tokens * per * 2, stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < pieces; i += stride) {
    const int64_t token = i / (2 * per);
    int piece = static_cast<int>(i - token * (2 * per));
    const bool value = piece >= per;
    piece -= value ? per : 0;
    const int row = a.rows[token];
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    float f = 1.0f;
    if (row >= 0 && row < a.cache_rows) {
      w = __ldcs(reinterpret_cast<const uint4*>((value ? a.v8 : a.k8) + static_cast<int64_t>(row) * a.hkv * 128) + piece);
      f = power_of_two(static_cast<int>((value ? a.v_exp : a.k_exp)[(piece >> 3) * a.ld_exp + row]) - 127);
    } else if (row >= a.cache_rows) {
      atomicCAS(&g_rotary_err, 0, kPackedBadLengths);
    }
    uint4* y = reinterpret_cast<uint4*>(value ? a.V + token * a.ld_v : a.K + token * a.ld_k) + 2 * piece;
    y[0] = make_uint4(bf16x2_of_e4m3x2(w.x, f), bf16x2_of_e4m3x2(w.x >> 16, f), bf16x2_of_e4m3x2(w.y, f), bf16x2_of_e4m3x2(w.y >> 16, f));
    y[1] = make_uint4(bf16x2_of_e4m3x2(w.z, f), bf16x2_of_e4m3x2(w.z >> 16, f), bf16x2_of_e4m3x2(w.w, f), bf16x2_of_e4m3x2(w.w >> 16, f));
  }
}

// Warps that share a token's groups of heads: one, or with few tokens as many as fill the GPU.
int token_split(int64_t tokens, int groups, int sms) {
  const int64_t want = (static_cast<int64_t>(sms) * 32 + tokens - 1) / (tokens > 0 ? tokens : 1);
  return static_cast<int>(want < 1 ? 1 : want > groups ? groups : want);
}
int groups_of(int heads) { return (heads + kHeadsAbreast - 1) / kHeadsAbreast; }

constexpr int kFwdBlocks = 8, kBwdBlocks = 4;  // blocks of an SM, at most

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int sms, cudaStream_t st) {
  const bool cache = a.rows != nullptr, norm = a.wq != nullptr || a.wk != nullptr, half = a.layout == 0;
  const int split = token_split(a.tokens, groups_of(a.hq) + (cache ? 2 : 1) * groups_of(a.hkv), sms);
  const int64_t blocks = (a.tokens * split + kWarps - 1) / kWarps, most = static_cast<int64_t>(sms) * kFwdBlocks;
  const dim3 grid(static_cast<unsigned>(blocks < most ? blocks : most));
  auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(kThreads), 0, 1, st, a, split); };
  if (cache)
    return norm ? (half ? go(rotary_kernel<true, true, true>) : go(rotary_kernel<true, false, true>))
                : (half ? go(rotary_kernel<false, true, true>) : go(rotary_kernel<false, false, true>));
  return norm ? (half ? go(rotary_kernel<true, true, false>) : go(rotary_kernel<true, false, false>))
              : (half ? go(rotary_kernel<false, true, false>) : go(rotary_kernel<false, false, false>));
}

int rotary_bwd_blocks(int64_t tokens, int hq, int hkv, int sms) {
  const int split = token_split(tokens, groups_of(hq) + groups_of(hkv), sms);
  const int64_t blocks = (tokens * split + kWarps - 1) / kWarps, most = static_cast<int64_t>(sms) * kBwdBlocks;
  return static_cast<int>(blocks < most ? blocks : most);
}

cudaError_t launch_rotary_bwd(const RotaryBwdArgs& a, float* part, int sms, cudaStream_t st) {
  const int split = token_split(a.tokens, groups_of(a.hq) + groups_of(a.hkv), sms);
  const dim3 grid(static_cast<unsigned>(rotary_bwd_blocks(a.tokens, a.hq, a.hkv, sms)));
  return a.layout == 0 ? launch_pdl(rotary_bwd_kernel<true>, grid, dim3(kThreads), 0, 1, st, a, part, split)
                       : launch_pdl(rotary_bwd_kernel<false>, grid, dim3(kThreads), 0, 1, st, a, part, split);
}

cudaError_t launch_rotary_sums(const RotaryBwdArgs& a, const float* part, int sms, cudaStream_t st) {
  const int blocks = a.tokens > 0 ? rotary_bwd_blocks(a.tokens, a.hq, a.hkv, sms) : 0;
  return launch_pdl(rotary_sums_kernel, dim3(8), dim3(256), 0, 1, st, a, part, blocks);
}

cudaError_t launch_cache_read(const CacheReadArgs& a, int sms, cudaStream_t st) {
  const int64_t blocks = (a.tokens * a.hkv * 16 + 255) / 256, most = static_cast<int64_t>(sms) * 8;
  return launch_pdl(cache_read_kernel, dim3(static_cast<unsigned>(blocks < most ? blocks : most)), dim3(256), 0, 1, st, a);
}

cudaError_t take_rotary_error(int* code) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_rotary_err, sizeof(int));
  if (e != cudaSuccess) return e;
  *code = v;
  if (v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_rotary_err, &zero, sizeof(int));
  }
  return e;
}

}  // namespace dm
