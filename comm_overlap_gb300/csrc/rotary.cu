// rotary.cu -- what stands between the fused projection and the attention: the norm of each query and key head with the
// rotation by position (forward, backward), and the 8-bit cache of keys and values (written in the same pass, read back).
//
// A head's 128 values are held by 8 lanes of a warp, two 16-byte pieces each, chosen so that a rotated pair always lies in one
// lane: with rot = 16 m rotated values, lane j < m holds pieces j and j + m (half layout: value i pairs with i + rot / 2, which
// is m pieces further; interleaved: 2 i with 2 i + 1, in one piece), the lanes from m on two neighbouring pieces of the rest.
// A warp takes twice four heads at a time, all of one token, whose cosines and sines it computes once.  Steps come through a ring in
// shared memory of each warp, several ahead, whatever token they belong to; it waits for no other warp.  Blocks are dealt to the kinds of
// heads by their bytes: forward, queries and keys have the same blocks and values others; backward each kind has its own, so that a
// lane keeps one kind's weight and sums in registers.
//
// Angles: a position turns pair i by position x frequency.  The frequency is kept as a 64-bit fraction of a turn, so the
// product's low 64 bits are the angle's fraction of a turn without any rounding by the position's size; what they are off the
// nearest quarter turn goes to sincospif.
//
// Bound: memory.  Forward 4 bytes a value, backward 6 (4 without norm), cache 3.  16384 tokens of 32 query and 8 key heads with norm: forward
// 57.7 us (5.8 TB/s, as a copy of the same bytes; 69 with loads into registers a step ahead), backward 82.6 (6.1), into the cache 64.9 (369 MB, 5.7);
// 147456 rows of 8 heads read back 142.5 (906 MB, 6.4).
#include <atomic>

#include "actfn.cuh"
#include "f32x2.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace dm {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kHeadsAbreast = 4;  // a warp's step has twice as many: with one four at a time the address and loop work weighs as much as the heads'
constexpr int kReadAbreast = 2;   // pieces of a lane in flight: with 4 a token of 8 heads leaves half the lanes idle
// Blocks of an SM and steps in the ring of a warp: the registers that two halves of a step take, and rings of 192 KB on an SM, of which one
// step is being read and 168 KB (backward 144) are in flight (96 KB and 64 for the cache, whose blocks wait less for memory than for the
// conversions).
constexpr int kFwdBlocks = 3, kFwdDepth = 8, kWriteBlocks = 4, kWriteDepth = 3, kBwdBlocks = 3, kBwdDepth = 4;
// Blocks of two kinds of heads, and the warps that share a token's steps.
struct RotaryShares {
  int blocks[2], split[2];
};
__host__ __device__ constexpr int steps_of(int heads) { return (heads + 2 * kHeadsAbreast - 1) / (2 * kHeadsAbreast); }

__device__ int g_rotary_err;

__device__ __forceinline__ void unpack8(const uint4& w, uint64_t (&v)[4]) {
  v[0] = f2(bf16lo(w.x), bf16hi(w.x));
  v[1] = f2(bf16lo(w.y), bf16hi(w.y));
  v[2] = f2(bf16lo(w.z), bf16hi(w.z));
  v[3] = f2(bf16lo(w.w), bf16hi(w.w));
}
__device__ __forceinline__ uint32_t pack2(uint64_t v) {
  float lo, hi;
  f2_split(v, lo, hi);
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ uint4 pack8(const uint64_t (&v)[4]) { return make_uint4(pack2(v[0]), pack2(v[1]), pack2(v[2]), pack2(v[3])); }
__device__ __forceinline__ float sum2(uint64_t v) {
  float lo, hi;
  f2_split(v, lo, hi);
  return lo + hi;
}

// Frequency (radians a position) as a fraction of a turn, in units of 2^-64 turns.
__device__ __forceinline__ unsigned long long turn_fraction(double f) {
  double t = f * 0.15915494309189533577;
  t -= floor(t);
  return __double2ull_rn(t * 18446744073709551616.0);
}

// The rotated pairs' turns a position, and 1 for each (NaN for a frequency that is not finite), by the first rot / 2 threads.
struct Turns {
  unsigned long long of[64];
  float one[64];
  __device__ __forceinline__ void load(const double* frequencies, int rot) {
    const int i = static_cast<int>(threadIdx.x);
    if (i >= (rot >> 1)) return;
    const double f = frequencies[i];
    of[i] = turn_fraction(f);
    one[i] = (__double2hiint(f) & 0x7FF00000) != 0x7FF00000 ? 1.0f : NAN;  // (fp64 arithmetic is slow here, and the blocks wait for it)
  }
};

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

// Cosines and sines of a token's angles, times the amplitude (and sines times `sign`), computed by the warp's lanes, two pairs each,
// to shared memory (64 of each a warp).
__device__ __forceinline__ void token_angles(float* cosines, float* sines, const Turns& turns, int position, int rot, float amplitude,
                                             float sign, int lane) {
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    if (i < (rot >> 1)) {
      const unsigned long long at = turns.of[i] * static_cast<unsigned long long>(static_cast<long long>(position));
      // the nearest quarter turn, and the rest, all of its 64 bits: an angle next to a quarter turn (or to none) keeps fp32's digits for itself
      const uint32_t quarter = static_cast<uint32_t>((at + (1ull << 61)) >> 62);
      float x, y;
      sincospif(static_cast<float>(static_cast<long long>(at - (static_cast<unsigned long long>(quarter) << 62))) * 0x1p-63f, &y, &x);
      const float cs = quarter & 1 ? (quarter & 2 ? y : -y) : (quarter & 2 ? -x : x);
      const float sn = quarter & 1 ? (quarter & 2 ? -x : x) : (quarter & 2 ? -y : y);
      const float size = amplitude * turns.one[i];
      cosines[i] = cs * size;
      sines[i] = sn * (size * sign);
    }
  }
  __syncwarp();
}
// Those of the lane's own pairs: half layout 8 j + e for (a[e], b[e]); interleaved 4 ca + i for (a[2 i], a[2 i + 1]) and 4 cb + i for b's.
template <bool HALF>
__device__ __forceinline__ void own_pairs(const float* v, const Place& p, uint64_t (&x)[4]) {
  const int first = HALF ? 8 * p.j : 4 * p.ca, second = HALF ? 8 * p.j + 4 : 4 * p.cb;
  const float4 y = *reinterpret_cast<const float4*>(v + first), z = *reinterpret_cast<const float4*>(v + second);
  x[0] = f2(y.x, y.y);
  x[1] = f2(y.z, y.w);
  x[2] = f2(z.x, z.y);
  x[3] = f2(z.z, z.w);
}

// (a, b) -> (a cos - b sin, a sin + b cos): half layout two pairs at a time, interleaved within each two values.
template <bool HALF>
__device__ __forceinline__ void rotate(uint64_t (&a)[4], uint64_t (&b)[4], const uint64_t (&c)[4], const uint64_t (&s)[4]) {
  if (HALF) {
    const uint64_t minus = f2(-1.0f, -1.0f);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint64_t x = a[e], y = b[e], ys = mul_f2(y, s[e]);
      a[e] = fma_f2(ys, minus, mul_f2(x, c[e]));
      b[e] = fma_f2(x, s[e], mul_f2(y, c[e]));
    }
  } else {
    auto turn = [](uint64_t& v, float cs, float sn) {
      float x, y;
      f2_split(v, x, y);
      v = f2(fmaf(x, cs, -y * sn), fmaf(x, sn, y * cs));
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float c0, c1, s0, s1;
      f2_split(c[i], c0, c1);
      f2_split(s[i], s0, s1);
      turn(a[2 * i], c0, s0);
      turn(a[2 * i + 1], c1, s1);
      f2_split(c[i + 2], c0, c1);
      f2_split(s[i + 2], s0, s1);
      turn(b[2 * i], c0, s0);
      turn(b[2 * i + 1], c1, s1);
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

constexpr float kInvD = 1.0f / 128.0f;
// Heads whose squares leave fp32's range are measured times this.
constexpr float kSmaller = 0x1p-80f;

// 1 / sqrt(mean(x^2) + eps) of the head, whose values are brought into range: x was multiplied by `small`, and so is the result.  To the
// nearest for what goes to 8 bits, where the last bit of fp32 can turn a value over to the next step.
__device__ __forceinline__ float head_rstd(uint64_t (&a)[4], uint64_t (&b)[4], float eps, float& small, bool nearest = false) {
  auto squares = [&] {
    uint64_t s0 = mul_f2(a[0], a[0]), s1 = mul_f2(b[0], b[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) {
      s0 = fma_f2(a[e], a[e], s0);
      s1 = fma_f2(b[e], b[e], s1);
    }
    return head_sum(sum2(add_f2(s0, s1)));
  };
  float ss = squares();
  small = 1.0f;
  if (__any_sync(0xFFFFFFFFu, !(ss < INFINITY))) {
    small = ss < INFINITY ? 1.0f : kSmaller;
    const uint64_t f = f2(small, small);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] = mul_f2(a[e], f);
      b[e] = mul_f2(b[e], f);
    }
    ss = squares();
  }
  const float mean = fmaf(ss, kInvD, eps * small * small);
  const float r = rsqrtf(mean);
  if (!nearest) return r;
  // a step of Newton's method, its residual 1 - mean r^2 from products without rounding
  const float h = mean * r, l = fmaf(mean, r, -h), e = fmaf(-l, r, fmaf(-h, r, 1.0f));
  return e == e ? fmaf(0.5f * r, e, r) : r;  // (an infinity has none)
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
__device__ __forceinline__ int quantise(const uint64_t (&a)[4], const uint64_t (&b)[4], uint2& qa, uint2& qb) {
  float x[8], y[8], amax = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f2_split(a[e], x[2 * e], x[2 * e + 1]);
    f2_split(b[e], y[2 * e], y[2 * e + 1]);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(fabsf(x[e]), fabsf(y[e])));
  amax = head_max(amax);
  if (__any_sync(0xFFFFFFFFu, !(amax < INFINITY))) {
    amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = fabsf(x[e]) < INFINITY ? x[e] : NAN;
      y[e] = fabsf(y[e]) < INFINITY ? y[e] : NAN;
      amax = fmaxf(amax, fmaxf(fabsf(x[e]), fabsf(y[e])));  // (NaN is passed over)
    }
    amax = head_max(amax);
  }
  const uint32_t bits = __float_as_uint(amax);
  int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u);
  e = amax > 0.0f ? min(max(e, -kCacheExpMax), kCacheExpMax) : 0;
  const float f = power_of_two(-e);
  qa = make_uint2(e4m3x4(x[0] * f, x[1] * f, x[2] * f, x[3] * f), e4m3x4(x[4] * f, x[5] * f, x[6] * f, x[7] * f));
  qb = make_uint2(e4m3x4(y[0] * f, y[1] * f, y[2] * f, y[3] * f), e4m3x4(y[4] * f, y[5] * f, y[6] * f, y[7] * f));
  return e;
}

// 16 bytes from memory to shared memory, zeros unless `there`; each lane reads back only what it asked for itself.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ int64_t divide(int64_t x, int y) {  // x >= 0; nearly always within 32 bits
  if ((x >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}
// A warp's way through its units: a unit is a token's steps (of twice four heads), or, with few tokens, every split-th of them.
struct Walk {
  int64_t unit, token;
  int step;
  __device__ __forceinline__ void enter(int64_t u, int64_t units, int split) {
    unit = u;
    if (u >= units) return;
    token = split == 1 ? u : divide(u, split);
    step = static_cast<int>(u - token * split);
  }
  // The next step; true where a unit begins.
  __device__ __forceinline__ bool next(int steps, int split, int64_t stride, int64_t units) {
    step += split;
    if (step < steps) return false;
    enter(unit + stride, units, split);
    return true;
  }
};

// What a lane multiplies its values with: half layout a' = a[..] A - b[..] B, b' = a C + b D, two pairs at a time (without norm A = D and
// B = C); interleaved the same for the two values of a pair, a's four pairs in the first two of each array.  Lanes that do not turn: a A
// and b D alone.
template <bool HALF>
__device__ __forceinline__ void turn_pairs(uint64_t (&a)[4], uint64_t (&b)[4], const uint64_t (&A)[4], const uint64_t (&B)[4],
                                           const uint64_t (&C)[4], const uint64_t (&D)[4]) {
  if (HALF) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint64_t x = a[e], y = b[e];
      a[e] = fma_f2(x, A[e], mul_f2(y, B[e]));  // (B is negative)
      b[e] = fma_f2(x, C[e], mul_f2(y, D[e]));
    }
  } else {
    auto turn = [](uint64_t& v, uint64_t A, uint64_t B, uint64_t C, uint64_t D, int half) {
      float x, y, k[4][2];
      f2_split(v, x, y);
      f2_split(A, k[0][0], k[0][1]);
      f2_split(B, k[1][0], k[1][1]);
      f2_split(C, k[2][0], k[2][1]);
      f2_split(D, k[3][0], k[3][1]);
      v = f2(fmaf(x, k[0][half], y * k[1][half]), fmaf(x, k[2][half], y * k[3][half]));
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      turn(a[2 * i], A[i], B[i], C[i], D[i], 0);
      turn(a[2 * i + 1], A[i], B[i], C[i], D[i], 1);
      turn(b[2 * i], A[i + 2], B[i + 2], C[i + 2], D[i + 2], 0);
      turn(b[2 * i + 1], A[i + 2], B[i + 2], C[i + 2], D[i + 2], 1);
    }
  }
}

// ---- forward
template <bool NORM, bool HALF, bool CACHE>
__global__ void __launch_bounds__(kThreads, CACHE ? kWriteBlocks : kFwdBlocks) rotary_kernel(const RotaryArgs a, const RotaryShares shares) {
  constexpr int kDepth = CACHE ? kWriteDepth : kFwdDepth;
  extern __shared__ __align__(16) uint8_t ring_all[];  // of each warp, kDepth steps of 2048 bytes
  __shared__ Turns turns;
  __shared__ __align__(16) float cosines[kWarps][64], sines[kWarps][64];
  pdl_launch();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool value = CACHE && static_cast<int>(blockIdx.x) >= shares.blocks[0];  // blocks of values come after the others
  const int place = static_cast<int>(blockIdx.x) - (value ? shares.blocks[0] : 0), split = shares.split[value];
  if (!value) turns.load(a.frequencies, a.rot);
  __syncthreads();
  const Place p = place_of(lane, a.rot);
  // steps of a token: of queries, then keys (or of values alone)
  const int q_steps = value ? 0 : steps_of(a.hq), steps = q_steps + steps_of(a.hkv);
  const int64_t units = a.tokens * split, stride = static_cast<int64_t>(shares.blocks[value]) * kWarps;
  Walk now, ahead;
  now.enter(static_cast<int64_t>(place) * kWarps + warp, units, split);
  if (now.unit >= units) return;
  ahead = now;
  const uint16_t* const k_from = (value ? a.V : a.K) + p.slot * 128;
  const int64_t k_ld = value ? a.ld_v : a.ld_k;
  const uint32_t ring = smem_u32(ring_all) + warp * (kDepth * 2048u) + lane * 16u;
  uint32_t fill = 0, take = 0;
  auto load = [&] {
    if (ahead.unit < units) {
      const bool query = ahead.step < q_steps;
      const int head = (ahead.step - (query ? 0 : q_steps)) * (2 * kHeadsAbreast) + p.slot, left = (query ? a.hq : a.hkv) - head;
      const uint16_t* x = query ? a.Q + ahead.token * a.ld_q + p.slot * 128 : k_from + ahead.token * k_ld;
      if (left > 0) x += (head - p.slot) * 128;  // (past the last head nothing is read)
      const uint4* v = reinterpret_cast<const uint4*>(x);
      const uint32_t to = ring + fill;
      copy16(to, v + p.ca, left > 0);
      copy16(to + 512u, v + p.cb, left > 0);
      if (left > kHeadsAbreast) {
        copy16(to + 1024u, v + kHeadsAbreast * 16 + p.ca, true);
        copy16(to + 1536u, v + kHeadsAbreast * 16 + p.cb, true);
      }
      ahead.next(steps, split, stride, units);
    }
    copies_commit();
    fill = fill + 2048u == kDepth * 2048u ? 0u : fill + 2048u;
  };
#pragma unroll 1
  for (int i = 0; i < kDepth - 1; ++i) load();
  // a token's position and cache row, loaded a unit before they are needed
  const bool turned = a.rot > 0 && !value;
  int position = 0, row = 0, to_row = 0;
  auto look = [&](int64_t unit) {
    if (unit >= units) return;
    const int64_t token = split == 1 ? unit : divide(unit, split);
    if (turned) position = a.positions[token];
    if (CACHE) row = a.rows[token];
  };
  look(now.unit);
  bool begins = true, was_query = false;
  uint64_t A[4], B[4], C[4], D[4];
  while (now.unit < units) {
    const bool query = now.step < q_steps;
    if (begins) {
      if (turned) token_angles(cosines[warp], sines[warp], turns, position, a.rot, a.amplitude, a.sign, lane);
      if (CACHE) {
        to_row = row;
        if (to_row >= a.cache_rows) {
          if (lane == 0) atomicCAS(&g_rotary_err, 0, kPackedBadLengths);
          to_row = -1;
        }
      }
      look(now.unit + stride);
    }
    if (!value && (begins || (NORM && query != was_query))) {
      // cosines and sines times the weights of what they are multiplied with
      if (p.turns) {
        own_pairs<HALF>(cosines[warp], p, A);
        own_pairs<HALF>(sines[warp], p, C);
        const uint64_t minus = f2(-1.0f, -1.0f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          D[e] = A[e];
          B[e] = mul_f2(C[e], minus);
        }
      }
      if (NORM) {
        const uint4* w = reinterpret_cast<const uint4*>(query ? a.wq : a.wk);
        uint64_t wa[4], wb[4];
        unpack8(w[p.ca], wa);
        unpack8(w[p.cb], wb);
        if (!p.turns) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            A[e] = wa[e];
            D[e] = wb[e];
          }
        } else if (HALF) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            A[e] = mul_f2(A[e], wa[e]);
            C[e] = mul_f2(C[e], wa[e]);
            B[e] = mul_f2(B[e], wb[e]);
            D[e] = mul_f2(D[e], wb[e]);
          }
        } else {  // the two weights of a pair lie side by side
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x0, y0, x1, y1;
            f2_split(e < 2 ? wa[2 * (e & 1)] : wb[2 * (e & 1)], x0, y0);
            f2_split(e < 2 ? wa[2 * (e & 1) + 1] : wb[2 * (e & 1) + 1], x1, y1);
            const uint64_t wx = f2(x0, x1), wy = f2(y0, y1);
            A[e] = mul_f2(A[e], wx);
            C[e] = mul_f2(C[e], wx);
            B[e] = mul_f2(B[e], wy);
            D[e] = mul_f2(D[e], wy);
          }
        }
      }
      was_query = query;
    }
    load();
    copies_wait<kDepth - 1>();
    const int heads = query ? a.hq : a.hkv, head0 = (now.step - (query ? 0 : q_steps)) * (2 * kHeadsAbreast) + p.slot;
    const uint32_t from = ring + take;
    take = take + 2048u == kDepth * 2048u ? 0u : take + 2048u;
    uint16_t* y = nullptr;
    if (!CACHE || query) y = (query ? a.Yq + now.token * a.ld_yq : a.Yk + now.token * a.ld_yk) + head0 * 128;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int head = head0 + half * kHeadsAbreast;
      if (half == 1 && head - p.slot >= heads) break;  // (the same in the whole warp)
      uint64_t va[4], vb[4];
      unpack8(ld_shared_v4(from + half * 1024u), va);
      unpack8(ld_shared_v4(from + half * 1024u + 512u), vb);
      if (!value) {
        float rstd = 1.0f;
        if (NORM) {
          float small;
          rstd = head_rstd(va, vb, a.eps, small, CACHE && !query);
        }
        if (p.turns) {
          turn_pairs<HALF>(va, vb, A, B, C, D);
        } else if (NORM) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            va[e] = mul_f2(va[e], A[e]);
            vb[e] = mul_f2(vb[e], D[e]);
          }
        }
        if (NORM) {
          const uint64_t r = f2(rstd, rstd);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            va[e] = mul_f2(va[e], r);
            vb[e] = mul_f2(vb[e], r);
          }
        }
      }
      if (CACHE && !query) {
        uint2 qa, qb;
        const int e = quantise(va, vb, qa, qb);
        if (to_row >= 0 && head < heads) {
          uint8_t* codes = (value ? a.v8 : a.k8) + (static_cast<int64_t>(to_row) * a.hkv + head) * 128;
          reinterpret_cast<uint2*>(codes)[p.ca] = qa;
          reinterpret_cast<uint2*>(codes)[p.cb] = qb;
          if (p.j == 0) (value ? a.v_exp : a.k_exp)[head * a.ld_exp + to_row] = static_cast<uint8_t>(e + 127);
        }
      } else if (head < heads) {
        uint4* to = reinterpret_cast<uint4*>(y + half * (kHeadsAbreast * 128));
        to[p.ca] = pack8(va);
        to[p.cb] = pack8(vb);
      }
    }
    begins = now.next(steps, split, stride, units);
  }
  copies_wait<0>();
}

// ---- backward with norm.  With u = amplitude R^T gy, n = x rstd: gx = rstd (u w - n mean(u w n)), gw = sum of u n over tokens
// and heads.  Each lane adds up its values' gw in registers over all its heads; a block leaves the 128 sums of its kind.
template <bool HALF>
__global__ void __launch_bounds__(kThreads, kBwdBlocks) rotary_bwd_kernel(const RotaryBwdArgs a, float* part, const RotaryShares shares) {
  extern __shared__ __align__(16) uint8_t ring_all[];  // of each warp, kBwdDepth steps of 4096 bytes
  __shared__ Turns turns;
  __shared__ __align__(16) float cosines[kWarps][64], sines[kWarps][64];
  __shared__ float sums[kWarps][128];
  pdl_launch();
  pdl_wait();
  turns.load(a.frequencies, a.rot);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kind = static_cast<int>(blockIdx.x) >= shares.blocks[0];  // 0 queries, 1 keys
  const int place = static_cast<int>(blockIdx.x) - (kind ? shares.blocks[0] : 0), split = shares.split[kind];
  const Place p = place_of(lane, a.rot);
  const int heads = kind == 0 ? a.hq : a.hkv, steps = steps_of(heads);
  const uint16_t* const gy = (kind == 0 ? a.gYq : a.gYk) + p.slot * 128;
  const uint16_t* const x = (kind == 0 ? a.Q : a.K) + p.slot * 128;
  uint16_t* const gx = (kind == 0 ? a.gQ : a.gK) + p.slot * 128;
  const int64_t ld_gy = kind == 0 ? a.ld_gyq : a.ld_gyk, ld_x = kind == 0 ? a.ld_q : a.ld_k, ld_gx = kind == 0 ? a.ld_gq : a.ld_gk;
  uint64_t wa[4], wb[4], acc[8];
  {
    const uint4* w = reinterpret_cast<const uint4*>(kind == 0 ? a.wq : a.wk);
    unpack8(w[p.ca], wa);
    unpack8(w[p.cb], wb);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = 0;
  const int64_t units = a.tokens * split, stride = static_cast<int64_t>(shares.blocks[kind]) * kWarps;
  Walk now, ahead;
  now.enter(static_cast<int64_t>(place) * kWarps + warp, units, split);
  ahead = now;
  const uint32_t ring = smem_u32(ring_all) + warp * (kBwdDepth * 4096u) + lane * 16u;
  uint32_t fill = 0, take = 0;
  auto load = [&] {
    if (ahead.unit < units) {
      const int head = ahead.step * (2 * kHeadsAbreast) + p.slot, left = heads - head;
      const int64_t in = left > 0 ? ahead.step * (2 * kHeadsAbreast * 128) : 0;
      const uint4* g = reinterpret_cast<const uint4*>(gy + ahead.token * ld_gy + in);
      const uint4* v = reinterpret_cast<const uint4*>(x + ahead.token * ld_x + in);
      const uint32_t to = ring + fill;
      copy16(to, g + p.ca, left > 0);
      copy16(to + 512u, g + p.cb, left > 0);
      copy16(to + 1024u, v + p.ca, left > 0);
      copy16(to + 1536u, v + p.cb, left > 0);
      if (left > kHeadsAbreast) {
        copy16(to + 2048u, g + kHeadsAbreast * 16 + p.ca, true);
        copy16(to + 2560u, g + kHeadsAbreast * 16 + p.cb, true);
        copy16(to + 3u * 1024u, v + kHeadsAbreast * 16 + p.ca, true);
        copy16(to + 3584u, v + kHeadsAbreast * 16 + p.cb, true);
      } else if (heads - (head - p.slot) > kHeadsAbreast) {  // others of the warp have a head there: zeros for the sums
        st_shared_v4(to + 2048u, 0u, 0u, 0u, 0u);
        st_shared_v4(to + 2560u, 0u, 0u, 0u, 0u);
        st_shared_v4(to + 3u * 1024u, 0u, 0u, 0u, 0u);
        st_shared_v4(to + 3584u, 0u, 0u, 0u, 0u);
      }
      ahead.next(steps, split, stride, units);
    }
    copies_commit();
    fill = fill + 4096u == kBwdDepth * 4096u ? 0u : fill + 4096u;
  };
#pragma unroll 1
  for (int i = 0; i < kBwdDepth - 1; ++i) load();
  int position = 0;
  auto look = [&](int64_t unit) {
    if (a.rot > 0 && unit < units) position = a.positions[split == 1 ? unit : divide(unit, split)];
  };
  look(now.unit);
  bool begins = true;
  uint64_t c[4], s[4];
  while (now.unit < units) {
    if (begins) {
      if (a.rot > 0) {
        token_angles(cosines[warp], sines[warp], turns, position, a.rot, a.amplitude, -1.0f, lane);
        if (p.turns) {
          own_pairs<HALF>(cosines[warp], p, c);
          own_pairs<HALF>(sines[warp], p, s);
        }
      }
      look(now.unit + stride);
    }
    load();
    copies_wait<kBwdDepth - 1>();
    const uint32_t from = ring + take;
    take = take + 4096u == kBwdDepth * 4096u ? 0u : take + 4096u;
    const int head0 = now.step * (2 * kHeadsAbreast) + p.slot;
    uint16_t* const y = gx + now.token * ld_gx + now.step * (2 * kHeadsAbreast * 128);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int head = head0 + half * kHeadsAbreast;
      if (half == 1 && head - p.slot >= heads) break;  // (the same in the whole warp)
      uint64_t ua[4], ub[4], xa[4], xb[4];
      unpack8(ld_shared_v4(from + half * 2048u), ua);
      unpack8(ld_shared_v4(from + half * 2048u + 512u), ub);
      unpack8(ld_shared_v4(from + half * 2048u + 1024u), xa);
      unpack8(ld_shared_v4(from + half * 2048u + 1536u), xb);
      if (p.turns) rotate<HALF>(ua, ub, c, s);
      float small;
      const float rstd = head_rstd(xa, xb, a.eps, small);
      const uint64_t r = f2(rstd, rstd);
      uint64_t dot = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        xa[e] = mul_f2(xa[e], r);
        xb[e] = mul_f2(xb[e], r);
        acc[e] = fma_f2(ua[e], xa[e], acc[e]);
        acc[4 + e] = fma_f2(ub[e], xb[e], acc[4 + e]);
        ua[e] = mul_f2(ua[e], wa[e]);
        ub[e] = mul_f2(ub[e], wb[e]);
        dot = fma_f2(ua[e], xa[e], dot);
        dot = fma_f2(ub[e], xb[e], dot);
      }
      const float m = -head_sum(sum2(dot)) * kInvD, f = rstd * small;
      const uint64_t mm = f2(m, m), ff = f2(f, f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ua[e] = mul_f2(ff, fma_f2(xa[e], mm, ua[e]));
        ub[e] = mul_f2(ff, fma_f2(xb[e], mm, ub[e]));
      }
      if (head < heads) {
        uint4* to = reinterpret_cast<uint4*>(y + half * (kHeadsAbreast * 128));
        to[p.ca] = pack8(ua);
        to[p.cb] = pack8(ub);
      }
    }
    begins = now.next(steps, split, stride, units);
  }
  copies_wait<0>();
  // over the warp's four heads, then the block's warps in order
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float v[2];
    f2_split(acc[e], v[0], v[1]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], 8);
      v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], 16);
      if (p.slot == 0) sums[warp][8 * (e < 4 ? p.ca : p.cb) + 2 * (e & 3) + i] = v[i];
    }
  }
  __syncthreads();
  float v = sums[0][threadIdx.x];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) v += sums[w][threadIdx.x];
  part[static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x] = v;
}

// The blocks' sums of a kind, added up in order by 32 rows of threads and then across them; one block for 32 columns of a kind.
__global__ void __launch_bounds__(1024) rotary_sums_kernel(const RotaryBwdArgs a, const float* part, const RotaryShares shares) {
  __shared__ float rows[32][33];
  pdl_launch();
  pdl_wait();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, kind = blockIdx.x >> 2, first_col = (blockIdx.x & 3) * 32;
  const int first = kind == 0 ? 0 : shares.blocks[0], last = first + shares.blocks[kind];
  float v = 0.0f;
#pragma unroll 8
  for (int b = first + y; b < last; b += 32) v += part[static_cast<int64_t>(b) * 128 + first_col + x];
  rows[y][x] = v;
  __syncthreads();
  v = rows[x][y];  // column y of the block's: its 32 partial sums lie in a warp
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  float* to = kind == 0 ? a.gwq : a.gwk;
  if (x == 0 && to) to[first_col + y] = a.accumulate ? to[first_col + y] + v : v;
}

// ---- cache, read back: a warp takes a token, a lane 8 codes of up to kReadAbreast pieces at a time
__device__ __forceinline__ uint32_t bf16x2_of_e4m3x2(uint16_t two, float f) {
  float lo, hi;
  asm("{\n\t.reg .b32 x;\n\t.reg .b16 l, h;\n\tcvt.rn.f16x2.e4m3x2 x, %2;\n\tmov.b32 {l, h}, x;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "h"(two));
  return pack_bf16x2(lo * f, hi * f);  // (exact)
}
__global__ void __launch_bounds__(256) cache_read_kernel(const CacheReadArgs a) {
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31, per = a.hkv * 16;  // pieces of a token in one of K and V
  const int64_t stride = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  int64_t token = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  int row = token < a.tokens ? a.rows[token] : 0;
  for (; token < a.tokens; token += stride) {
    const int next = token + stride < a.tokens ? a.rows[token + stride] : 0;
    const bool there = row >= 0 && row < a.cache_rows;
    if (row >= a.cache_rows && lane == 0) atomicCAS(&g_rotary_err, 0, kPackedBadLengths);
    const uint8_t* k8 = a.k8 + static_cast<int64_t>(row) * a.hkv * 128;
    const uint8_t* v8 = a.v8 + static_cast<int64_t>(row) * a.hkv * 128;
    for (int first = lane; first < 2 * per; first += 32 * kReadAbreast) {
      uint2 w[kReadAbreast];
      int e[kReadAbreast];
#pragma unroll
      for (int i = 0; i < kReadAbreast; ++i) {
        const int at = first + 32 * i, piece = at < per ? at : at - per;
        w[i] = make_uint2(0u, 0u);
        e[i] = 127;
        if (there && at < 2 * per) {
          w[i] = __ldcs(reinterpret_cast<const uint2*>(at < per ? k8 : v8) + piece);
          e[i] = (at < per ? a.k_exp : a.v_exp)[(piece >> 4) * a.ld_exp + row];
        }
      }
#pragma unroll
      for (int i = 0; i < kReadAbreast; ++i) {
        const int at = first + 32 * i, piece = at < per ? at : at - per;
        if (at >= 2 * per) break;
        const float f = power_of_two(e[i] - 127);
        reinterpret_cast<uint4*>(at < per ? a.K + token * a.ld_k : a.V + token * a.ld_v)[piece] =
            make_uint4(bf16x2_of_e4m3x2(static_cast<uint16_t>(w[i].x), f), bf16x2_of_e4m3x2(static_cast<uint16_t>(w[i].x >> 16), f),
                       bf16x2_of_e4m3x2(static_cast<uint16_t>(w[i].y), f), bf16x2_of_e4m3x2(static_cast<uint16_t>(w[i].y >> 16), f));
      }
    }
    row = next;
  }
}

// Two kinds of blocks with so many steps a token each: by their steps, at most sms x blocks_of_sm altogether; one warp takes a token's
// steps, or with few tokens as many as fill the GPU.  Both kinds should end together.  Backward both compute a token's angles, which counts as
// `more` halves of a step (16384 tokens of 32 query and 8 key heads 86 us; 96 without, 89 with a quarter, 88 with three).  Into the cache
// values go through the tokens beside the queries and keys of the same rows, by their steps alone: 65 us, with a tenth more or fewer
// blocks 67 - 71.
RotaryShares shares_of(int64_t tokens, int steps0, int steps1, int more, int sms, int blocks_of_sm) {
  const int steps[2] = {steps0, steps1}, most = sms * blocks_of_sm;
  const int cost0 = steps0 ? 2 * steps0 + more : 0, cost1 = steps1 ? 2 * steps1 + more : 0;
  RotaryShares s = {};
  int left = most;
  for (int i = 1; i >= 0; --i) {
    if (steps[i] == 0 || tokens == 0) continue;
    const int64_t want = (int64_t(sms) * 16 + tokens - 1) / tokens;
    s.split[i] = static_cast<int>(want > steps[i] ? steps[i] : want);
    const int64_t units = (tokens * s.split[i] + kWarps - 1) / kWarps;
    int share = i == 0 ? left : static_cast<int>((int64_t(most) * cost1 + (cost0 + cost1) / 2) / (cost0 + cost1));
    if (share < 1) share = 1;
    if (i == 1 && steps0 > 0 && share >= most) share = most - 1;
    s.blocks[i] = static_cast<int>(units < share ? units : share);
    left -= s.blocks[i];
  }
  return s;
}
// The opt-in to more than 48 KB of shared memory, once for each kernel and device.
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<bool> (&ready)[kMaxDevices]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (ready[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) ready[dev].store(true, std::memory_order_release);
  return e;
}

RotaryShares fwd_shares(int64_t tokens, int hq, int hkv, bool values, int sms) {
  return shares_of(tokens, steps_of(hq) + steps_of(hkv), values ? steps_of(hkv) : 0, 0, sms, values ? kWriteBlocks : kFwdBlocks);
}
RotaryShares bwd_shares(int64_t tokens, int hq, int hkv, int sms) {
  return shares_of(tokens, steps_of(hq), steps_of(hkv), 1, sms, kBwdBlocks);
}

template <bool NORM, bool HALF, bool CACHE>
cudaError_t launch_fwd(const RotaryArgs& a, const RotaryShares& s, cudaStream_t st) {
  static std::atomic<bool> ready[kMaxDevices];
  constexpr int kBytes = kWarps * 2048 * (CACHE ? kWriteDepth : kFwdDepth);
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(rotary_kernel<NORM, HALF, CACHE>), kBytes, ready);
  if (e != cudaSuccess) return e;
  return launch_pdl(rotary_kernel<NORM, HALF, CACHE>, dim3(static_cast<unsigned>(s.blocks[0] + s.blocks[1])), dim3(kThreads), size_t(kBytes), 1,
                    st, a, s);
}
template <bool HALF>
cudaError_t launch_bwd(const RotaryBwdArgs& a, float* part, const RotaryShares& s, cudaStream_t st) {
  static std::atomic<bool> ready[kMaxDevices];
  constexpr int kBytes = kWarps * 4096 * kBwdDepth;
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(rotary_bwd_kernel<HALF>), kBytes, ready);
  if (e != cudaSuccess) return e;
  return launch_pdl(rotary_bwd_kernel<HALF>, dim3(static_cast<unsigned>(s.blocks[0] + s.blocks[1])), dim3(kThreads), size_t(kBytes), 1, st, a,
                    part, s);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int sms, cudaStream_t st) {
  const bool cache = a.rows != nullptr, norm = a.wq != nullptr || a.wk != nullptr, half = a.layout == 0;
  const RotaryShares s = fwd_shares(a.tokens, a.hq, a.hkv, cache, sms);
  if (cache)
    return norm ? (half ? launch_fwd<true, true, true>(a, s, st) : launch_fwd<true, false, true>(a, s, st))
                : (half ? launch_fwd<false, true, true>(a, s, st) : launch_fwd<false, false, true>(a, s, st));
  return norm ? (half ? launch_fwd<true, true, false>(a, s, st) : launch_fwd<true, false, false>(a, s, st))
              : (half ? launch_fwd<false, true, false>(a, s, st) : launch_fwd<false, false, false>(a, s, st));
}

int rotary_bwd_blocks(int64_t tokens, int hq, int hkv, int sms) {
  const RotaryShares s = bwd_shares(tokens, hq, hkv, sms);
  return s.blocks[0] + s.blocks[1];
}

cudaError_t launch_rotary_bwd(const RotaryBwdArgs& a, float* part, int sms, cudaStream_t st) {
  const RotaryShares s = bwd_shares(a.tokens, a.hq, a.hkv, sms);
  return a.layout == 0 ? launch_bwd<true>(a, part, s, st) : launch_bwd<false>(a, part, s, st);
}

cudaError_t launch_rotary_sums(const RotaryBwdArgs& a, const float* part, int sms, cudaStream_t st) {
  const RotaryShares s = bwd_shares(a.tokens, a.hq, a.hkv, sms);
  return launch_pdl(rotary_sums_kernel, dim3(8), dim3(1024), 0, 1, st, a, part, s);
}

cudaError_t launch_cache_read(const CacheReadArgs& a, int sms, cudaStream_t st) {
  const int64_t blocks = (a.tokens + 7) / 8, most = (int64_t(1) << 31) - 1;
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
