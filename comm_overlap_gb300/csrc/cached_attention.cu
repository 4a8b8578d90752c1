// cached_attention.cu -- attention of the last few tokens of each sequence over the 8-bit cache (rotary.cu writes it), and over
// rows that all sequences share.
//
// Keys and values are E4M3 codes with one power of two for each row and head, so K = k8 2^a and V = v8 2^b.  The scores are
// products of the codes times 2^a; with t = scale log2(e) q k + b and the running maximum m of t, a key weighs w = 2^(t - m) <= 1,
// which is its softmax weight times its value's 2^b: O = sum w v8, and the denominator is sum w 2^-b.  Codes convert to f16
// without rounding; q is scaled by a power of two for each row so that its largest value lies in [2^14, 2^15) and keeps its
// 8 bits down to 2^-24; w is rounded to f16 (11 bits), which is finer than the bf16 of the output.  Sums are fp32.
//
// A row of scores is a token and one of the `group` query heads of a key head.  Products are computed transposed, keys x rows
// (mma m16n8k16: 16 keys x 8 rows, then 16 elements x 8 rows), so that 8 rows, one token of up to 8 heads, fill an instruction,
// and a warp converts each code once.  A warp holds NT x 8 rows; `share` warps read the same tiles of 32 keys for more.
// tcgen05 would want 128 rows; here the conversions and memory bound the kernel, not the products.
//
// The tiles of all sequences and key heads, laid end to end, are cut into equal ranges, one for each stream of warps on the GPU.
// A stream loads its tiles by TMA into a ring of its own.  What covers all keys of a row is written out; parts leave their m,
// denominator and O in the workspace, and a second kernel joins them in order.
// Bound: memory, 2 x 129 bytes a key and key head.
#include <cuda_bf16.h>

#include <atomic>
#include <type_traits>

#include "actfn.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace dm {

namespace {

__device__ int g_cached_err;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kKeys = kCachedKeys;                 // of a tile
constexpr int kStages = 3;
constexpr uint32_t kTile = kKeys * 128;            // bytes of K or V
constexpr uint32_t kStage = 2 * kTile;
constexpr uint32_t kCtrl = 2048;
constexpr int kSmem = 1024 + static_cast<int>(kCtrl) + kWarps * kStages * static_cast<int>(kStage);
static_assert(kSmem <= 232448, "shared memory beyond the per-CTA limit");
constexpr int kSms = 152;                          // CTAs that the workspace is sized for, at most
constexpr int kPart = 132;                         // floats of a partial row: 128 of O, m, denominator, two unused

// ---- work: tiles of all items (sequence, block of rows, key head) in order

struct CachedHeader {
  int64_t tiles;    // of all items
  int64_t streams;  // ranges that they are cut into
};

struct CachedWork {
  CachedHeader* head;
  int64_t* base;    // tiles before each sequence
  float* slots;     // two for each stream: `rows` partial rows each
  float* whole;     // partial rows of items that were not cut, by token and head (with a shared prefix)
};

// First row and length of a sequence; one whose rows leave the cache gets none and is recorded.
__device__ __forceinline__ int sequence(const CachedArgs& a, int s, int& start) {
  start = a.k_start[s];
  int len = a.k_len[s];
  if (start < 0 || len < 0 || len > a.cache_rows || start > a.cache_rows - len) {
    atomicCAS(&g_cached_err, 0, kPackedBadLengths);
    start = len = 0;
  }
  return len;
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kKeys - 1) / kKeys; }

// Where stream i's range begins, and the stream that tile x belongs to.
__device__ __forceinline__ int64_t range_begin(int64_t i, const CachedHeader& h) { return i * h.tiles / h.streams; }
__device__ __forceinline__ int64_t stream_of(int64_t x, const CachedHeader& h) {
  return ((x + 1) * h.streams + h.tiles - 1) / h.tiles - 1;
}

struct Cursor {
  int s, start, len, tiles, item, tile;  // item: block of rows x hkv + key head, of sequence s
};

__device__ __forceinline__ void next_sequence(const CachedArgs& a, Cursor& c) {
  c.item = c.tile = 0;
  do {
    ++c.s;
    c.len = c.s < a.n ? sequence(a, c.s, c.start) : 0;
    c.tiles = tiles_of(c.len);
  } while (c.tiles == 0 && c.s < a.n);
}
__device__ __forceinline__ void next_item(const CachedArgs& a, Cursor& c) {
  c.tile = 0;
  if (++c.item == a.blocks * a.hkv) next_sequence(a, c);
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The two codes in the lower, or upper, half of w as f16.
__device__ __forceinline__ uint32_t f16_lower(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t f16_upper(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ uint32_t has_nan(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }
__device__ __forceinline__ uint32_t has_nan(const uint4& v) { return has_nan(v.x) | has_nan(v.y) | has_nan(v.z) | has_nan(v.w); }

// The tile's key that index x of an instruction's 8 stands for.  Of the rows of 128 bytes under the 128-byte swizzle (16-byte piece
// p of row r lies at p ^ (r mod 8)), K's loads take pieces 0 - 3 or 4 - 7 of rows key(2 i) and key(2 i + 1) at once, V's pieces 2 i and
// 2 i + 1 of rows key(0), key(2), key(4), key(6) or of the others: with this order neither meets a bank twice.
__device__ __forceinline__ int key_of(int x) { return x & 1 ? ((x - 1) ^ 4) + 1 : x; }

template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
    cached_attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const CachedArgs a,
                            const CachedWork w) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t ctrl = (smem_u32(smem_raw) + 1023u) & ~1023u, ring0 = ctrl + kCtrl;
  uint8_t* const ctrl_ptr = smem_raw + (ctrl - smem_u32(smem_raw));
  __shared__ int64_t before[kThreads + 1];  // tiles of one item before each thread's sequences
  __shared__ int64_t warp_sums[kWarps];
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ctrl_ptr + kCtrl - 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int stream_slot = warp / a.share, member = warp - stream_slot * a.share, slots = kWarps / a.share;
  const uint32_t bars = ctrl + 64u * static_cast<uint32_t>(stream_slot);
  const uint32_t ring = ring0 + static_cast<uint32_t>(stream_slot * kStages) * kStage;
  if (threadIdx.x == 0) *abort_flag = 0;
  if (member == 0 && lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(bars + 8u * i, 1);
    fence_mbar_init();
  }
  pdl_launch();
  pdl_wait();

  // ---- the plan, by every block for itself: tiles before each thread's range of sequences
  const int per = (a.n + kThreads - 1) / kThreads, s0 = min(static_cast<int>(threadIdx.x) * per, a.n), s1 = min(s0 + per, a.n);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) {
    int start;
    mine += tiles_of(sequence(a, s, start));
  }
  int64_t sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) warp_sums[warp] = sum;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i == warp) sum += total;
    total += warp_sums[i];
  }
  before[threadIdx.x] = sum - mine;
  if (threadIdx.x == 0) before[kThreads] = total;
  __syncthreads();
  const int64_t items = static_cast<int64_t>(a.blocks) * a.hkv;  // of a sequence
  CachedHeader h;
  h.tiles = total * items;
  {
    const int64_t most = static_cast<int64_t>(gridDim.x) * slots;
    h.streams = h.tiles < most ? (h.tiles > 0 ? h.tiles : 1) : most;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *w.head = h;
  if (threadIdx.x % gridDim.x == blockIdx.x) {  // for the second kernel
    int64_t at = (sum - mine) * items;
    for (int s = s0; s < s1; ++s) {
      int start;
      w.base[s] = at;
      at += static_cast<int64_t>(tiles_of(sequence(a, s, start))) * items;
    }
  }

  const int64_t stream = static_cast<int64_t>(stream_slot) * gridDim.x + blockIdx.x;
  if (stream >= h.streams || h.tiles == 0) return;  // (all warps of a stream)
  const int64_t lo = range_begin(stream, h), hi = range_begin(stream + 1, h);
  Cursor at;
  {
    // the thread whose sequences hold tile lo, then the sequence, 32 at a time
    int x = 0;
    for (int step = kThreads / 2; step > 0; step >>= 1)
      if (before[x + step] * items <= lo) x += step;
    int64_t done = before[x] * items;
    at.s = min(x * per, a.n);
    at.len = at.start = at.tiles = at.item = at.tile = 0;
    for (; at.s < a.n; at.s += 32) {
      int start = 0;
      const int len = at.s + lane < a.n ? sequence(a, at.s + lane, start) : 0;
      int64_t upto = tiles_of(len);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += v;
      }
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, done + upto * items > lo);
      if (past) {
        const int l = __ffs(past) - 1;
        at.len = __shfl_sync(0xFFFFFFFFu, len, l);
        at.start = __shfl_sync(0xFFFFFFFFu, start, l);
        at.tiles = tiles_of(at.len);
        done += (__shfl_sync(0xFFFFFFFFu, upto, l) - at.tiles) * items;
        at.s += l;
        break;
      }
      done += __shfl_sync(0xFFFFFFFFu, upto, 31) * items;
    }
    if (at.tiles > 0) {
      at.item = static_cast<int>((lo - done) / at.tiles);
      at.tile = static_cast<int>((lo - done) - static_cast<int64_t>(at.item) * at.tiles);
    }
  }

  // ---- loads: tile by tile, kStages ahead; the lanes keep their key's two exponents
  Cursor ahead = at;
  int64_t loads_left = hi - lo;
  int issued = 0;
  int exps[kStages];
  bool ok = true;
  auto load = [&]() -> int {
    if (loads_left == 0) return 0;
    --loads_left;
    const int head = ahead.item % a.hkv, row = ahead.start + ahead.tile * kKeys;
    if (member == 0 && elect_one() && ok) {
      const int stage = issued % kStages;
      const uint32_t bar = bars + 8u * stage, to = ring + static_cast<uint32_t>(stage) * kStage;
      mbar_arrive_expect_tx(bar, kStage);
      tma_load_3d(to, &map_k, bar, 0, head, row);
      tma_load_3d(to + kTile, &map_v, bar, 0, head, row);
    }
    ++issued;
    int e = 0;
    if (row + lane < a.cache_rows) {
      const int64_t x = head * a.ld_exp + row + lane;
      e = static_cast<int>(a.k_exp[x]) | static_cast<int>(a.v_exp[x]) << 8;
    }
    if (++ahead.tile == ahead.tiles) next_item(a, ahead);
    return e;
  };
#pragma unroll
  for (int i = 0; i < kStages; ++i) exps[i] = load();

  const int kg = key_of(g), ka = key_of(2 * c), kb = key_of(2 * c + 1);
  const uint32_t k_lo = kg * 128 + ((c ^ kg) << 4), k_hi = kg * 128 + (((c + 4) ^ kg) << 4);
  const uint32_t v_a = kTile + ka * 128 + ((g ^ ka) << 4), v_b = kTile + kb * 128 + ((g ^ kb) << 4);
  auto release = [&] {  // the stream's warps have read a tile
    if (a.share == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(stream_slot + 1), "r"(a.share * 32) : "memory");
  };
  int consumed = 0;
  for (int64_t x = lo; x < hi;) {
    if (at.s >= a.n) {  // (only where lengths change while the kernel reads them)
      for (; x < hi; ++x) release();
      break;
    }
    // ---- one item: rows block * rows .. of the sequence, keys of tiles at.tile .. last - 1
    const int block = at.item / a.hkv, head = at.item - block * a.hkv;
    const int last = static_cast<int>(min(static_cast<int64_t>(at.tiles), at.tile + (hi - x)));
    const int row0 = (block * a.share + member) * NT * 8, rows = a.t * a.group;
    const bool idle = row0 >= rows;
    uint32_t q[NT][8][2];
    float row_scale[NT][2];
    int limit[NT][2];
    int least = at.len;  // keys that every row of the warp sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + nt * 8 + g;
      float v[2][16];
      if (r < rows) {
        const int token = r / a.group;
        const uint16_t* p = a.Q + (static_cast<int64_t>(at.s) * a.t + token) * a.ld_q + (head * a.group + r - token * a.group) * 128;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint4* u = reinterpret_cast<const uint4*>(p + half * 64 + c * 16);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 y = u[i];
            v[half][8 * i + 0] = bf16lo(y.x); v[half][8 * i + 1] = bf16hi(y.x);
            v[half][8 * i + 2] = bf16lo(y.y); v[half][8 * i + 3] = bf16hi(y.y);
            v[half][8 * i + 4] = bf16lo(y.z); v[half][8 * i + 5] = bf16hi(y.z);
            v[half][8 * i + 6] = bf16lo(y.w); v[half][8 * i + 7] = bf16hi(y.w);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[0][i] = v[1][i] = 0.0f;
      }
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fmaxf(fabsf(v[0][i]), fabsf(v[1][i])));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      // 2^up brings the largest into [2^14, 2^15) (an infinity stays one)
      const int up = amax > 0.0f && amax < INFINITY ? min(14 + 127 - static_cast<int>(__float_as_uint(amax) >> 23), 120) : 0;
      const float f = __int_as_float((up + 127) << 23);
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const float* y = v[s >> 2] + 4 * (s & 3);
        q[nt][s][0] = pack_f16x2(y[0] * f, y[1] * f);
        q[nt][s][1] = pack_f16x2(y[2] * f, y[3] * f);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {  // this lane's columns: rows 2 c and 2 c + 1
        const int rj = row0 + nt * 8 + 2 * c + j;
        const int up_j = __shfl_sync(0xFFFFFFFFu, up, 4 * (2 * c + j));
        row_scale[nt][j] = a.scale_log2 * __int_as_float((127 - up_j) << 23);
        limit[nt][j] = a.causal && rj < rows ? at.len - a.t + rj / a.group + 1 : at.len;
        least = min(least, limit[nt][j]);
      }
    }
    least = __reduce_min_sync(0xFFFFFFFFu, least);
    float o[8][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[nt][j] = -INFINITY;
        l[nt][j] = 0.0f;
      }

    for (int tile = at.tile; tile < last; ++tile) {
      const int stage = consumed % kStages;
      const uint32_t kv = ring + static_cast<uint32_t>(stage) * kStage;
      ok = mbar_wait(bars + 8u * stage, (consumed / kStages) & 1, abort_flag, &g_cached_err, a.err_site) && ok;
      ++consumed;
      if (!idle) {
        const int key0 = tile * kKeys, e = key0 + lane < at.len ? exps[0] : 127 | 127 << 8;
        float acc[2][NT][4], key_scale[2][2], bias[2][2], unbias[2][2];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) acc[mt][nt][0] = acc[mt][nt][1] = acc[mt][nt][2] = acc[mt][nt][3] = 0.0f;
          const uint32_t p = kv + mt * 2048u;
          const uint4 x0 = ld_shared_v4(p + k_lo), x1 = ld_shared_v4(p + k_lo + 1024u);
          const uint4 y0 = ld_shared_v4(p + k_hi), y1 = ld_shared_v4(p + k_hi + 1024u);
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            const uint32_t u = word_of(s < 4 ? x0 : y0, s & 3), v = word_of(s < 4 ? x1 : y1, s & 3);
            const uint32_t a0 = f16_lower(u), a1 = f16_lower(v), a2 = f16_upper(u), a3 = f16_upper(v);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(acc[mt][nt], a0, a1, a2, a3, q[nt][s][0], q[nt][s][1]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {  // keys g and g + 8 of the instruction
            const int both = __shfl_sync(0xFFFFFFFFu, e, mt * 16 + i * 8 + kg), b = both >> 8;
            key_scale[mt][i] = __int_as_float((both & 255) << 23);
            bias[mt][i] = static_cast<float>(b - 127);
            unbias[mt][i] = __int_as_float((254 - b) << 23);
          }
        }
        const bool tail = key0 + kKeys > least;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float t = fmaf(acc[mt][nt][i] * key_scale[mt][i >> 1], row_scale[nt][i & 1], bias[mt][i >> 1]);
              if (tail && key0 + mt * 16 + (i >> 1) * 8 + kg >= limit[nt][i & 1]) t = -INFINITY;
              acc[mt][nt][i] = t;
            }
        // running maximum
        bool moved = false;
        float factor[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float top = fmaxf(fmaxf(acc[0][nt][j], acc[0][nt][2 + j]), fmaxf(acc[1][nt][j], acc[1][nt][2 + j]));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 16));
            top = fmaxf(top, m[nt][j]);
            factor[nt][j] = top == m[nt][j] ? 1.0f : ex2_approx(m[nt][j] - top);
            moved |= top != m[nt][j];
            m[nt][j] = top;
          }
        if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            l[nt][0] *= factor[nt][0];
            l[nt][1] *= factor[nt][1];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[i][nt][0] *= factor[nt][0];
              o[i][nt][1] *= factor[nt][1];
              o[i][nt][2] *= factor[nt][0];
              o[i][nt][3] *= factor[nt][1];
            }
          }
        }
        uint32_t p[2][NT][2];  // weights in f16, rows 2 c and 2 c + 1, of keys g and g + 8
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float m0 = m[nt][0] == -INFINITY ? 0.0f : m[nt][0], m1 = m[nt][1] == -INFINITY ? 0.0f : m[nt][1];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float w0 = ex2_approx(acc[mt][nt][2 * i] - m0), w1 = ex2_approx(acc[mt][nt][2 * i + 1] - m1);
              l[nt][0] = fmaf(w0, unbias[mt][i], l[nt][0]);
              l[nt][1] = fmaf(w1, unbias[mt][i], l[nt][1]);
              p[mt][nt][i] = pack_f16x2(w0, w1);
            }
        }
        // O += V^T P; `only`: for the rows that see `sees` keys alone (a weight of zero times NaN must not reach the others)
        auto add_values = [&](int mt, const uint4& xa, const uint4& xb, const uint4& ya, const uint4& yb, auto only, int sees) {
          uint32_t b[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            b[nt][0] = transposed(p[mt][nt][0]);
            b[nt][1] = transposed(p[mt][nt][1]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t sel = i & 1 ? 0x7362u : 0x5140u;
            const uint32_t u = __byte_perm(word_of(xa, i >> 1), word_of(xb, i >> 1), sel);
            const uint32_t v = __byte_perm(word_of(ya, i >> 1), word_of(yb, i >> 1), sel);
            const uint32_t a0 = f16_lower(u), a1 = f16_upper(u), a2 = f16_lower(v), a3 = f16_upper(v);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float k0 = o[i][nt][0], k1 = o[i][nt][1], k2 = o[i][nt][2], k3 = o[i][nt][3];
              mma16816(o[i][nt], a0, a1, a2, a3, b[nt][0], b[nt][1]);
              if (decltype(only)::value) {
                if (limit[nt][0] != sees) {
                  o[i][nt][0] = k0;
                  o[i][nt][2] = k2;
                }
                if (limit[nt][1] != sees) {
                  o[i][nt][1] = k1;
                  o[i][nt][3] = k3;
                }
              }
            }
          }
        };
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const uint32_t at_v = kv + mt * 2048u;
          uint4 xa = ld_shared_v4(at_v + v_a), xb = ld_shared_v4(at_v + v_b);
          uint4 ya = ld_shared_v4(at_v + v_a + 1024u), yb = ld_shared_v4(at_v + v_b + 1024u);
          if (tail) {
            const int k0 = key0 + mt * 16;
            if (k0 + ka >= at.len) xa = zero;  // what lies past the sequence's keys has no effect, NaN included
            if (k0 + kb >= at.len) xb = zero;
            if (k0 + ka + 8 >= at.len) ya = zero;
            if (k0 + kb + 8 >= at.len) yb = zero;
            // NaN among values that some rows see and some do not: each token's rows by themselves
            if (least < at.len && __any_sync(0xFFFFFFFFu, has_nan(xa) | has_nan(xb) | has_nan(ya) | has_nan(yb))) {
              const int first = row0 / a.group, end = (min(row0 + NT * 8, rows) - 1) / a.group;
              for (int token = first; token <= end; ++token) {
                const int sees = at.len - a.t + token + 1;
                add_values(mt, k0 + ka < sees ? xa : zero, k0 + kb < sees ? xb : zero, k0 + ka + 8 < sees ? ya : zero,
                           k0 + kb + 8 < sees ? yb : zero, std::true_type(), sees);
              }
              continue;
            }
          }
          add_values(mt, xa, xb, ya, yb, std::false_type(), 0);
        }
      }
      release();  // the tile's place takes the next one
#pragma unroll
      for (int i = 0; i + 1 < kStages; ++i) exps[i] = exps[i + 1];
      exps[kStages - 1] = load();
    }

    // ---- what the item's keys came to
    const bool all = at.tile == 0 && last == at.tiles;
    x += last - at.tile;
    if (!idle && ok) {
      const int64_t begin = x - last;  // the item's first tile
      float* slot = w.slots + (2 * stream + (begin > lo ? 1 : 0)) * (static_cast<int64_t>(a.share) * NT * 8 * kPart);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float den = l[nt][j];
          den += __shfl_xor_sync(0xFFFFFFFFu, den, 4);
          den += __shfl_xor_sync(0xFFFFFFFFu, den, 8);
          den += __shfl_xor_sync(0xFFFFFFFFu, den, 16);
          const int in_warp = nt * 8 + 2 * c + j, r = row0 + in_warp;
          if (r >= rows) continue;
          const int token = r / a.group;
          const int64_t row = static_cast<int64_t>(at.s) * a.t + token;
          const int qh = head * a.group + r - token * a.group;
          if (all && !a.partial) {
            const bool some = den > 0.0f || den != den;
            const float inv = some ? 1.0f / den : 0.0f;
            uint4* y = reinterpret_cast<uint4*>(a.O + row * a.ld_o + static_cast<int64_t>(qh) * 128 + 16 * g);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              y[i] = make_uint4(pack_bf16x2(o[4 * i][nt][j] * inv, o[4 * i][nt][2 + j] * inv),
                                pack_bf16x2(o[4 * i + 1][nt][j] * inv, o[4 * i + 1][nt][2 + j] * inv),
                                pack_bf16x2(o[4 * i + 2][nt][j] * inv, o[4 * i + 2][nt][2 + j] * inv),
                                pack_bf16x2(o[4 * i + 3][nt][j] * inv, o[4 * i + 3][nt][2 + j] * inv));
            if (g == 0 && a.lse) a.lse[row * a.hq + qh] = some ? (m[nt][j] + log2f(den)) * 0.69314718055994531f : -INFINITY;
          } else {
            float* y = all ? w.whole + (row * a.hq + qh) * kPart : slot + (member * NT * 8 + in_warp) * kPart;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<float4*>(y + 16 * g + 4 * i) =
                  make_float4(o[2 * i][nt][j], o[2 * i][nt][2 + j], o[2 * i + 1][nt][j], o[2 * i + 1][nt][2 + j]);
            if (g == 0) *reinterpret_cast<float2*>(y + 128) = make_float2(m[nt][j], den);
          }
        }
    }
    at.tile = last;
    if (last == at.tiles) next_item(a, at);
  }
  if (!ok) {  // after a wait that ran out: copies in flight land before the block leaves
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 100000ull) {
    }
  }
}

// ---- join: a warp for each row (token and head); lane i has elements 4 i .. 4 i + 3
// (A part without a maximum still counts: its keys may all be NaN.)
struct Joined {
  float m = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  __device__ __forceinline__ void add(const float* part, int lane) {
    const float2 ml = *reinterpret_cast<const float2*>(part + 128);
    const float4 v = *reinterpret_cast<const float4*>(part + 4 * lane);
    const float top = fmaxf(m, ml.x);
    const float f = m == top ? 1.0f : ex2_approx(m - top), e = ml.x == top ? 1.0f : ex2_approx(ml.x - top);
    m = top;
    l = l * f + ml.y * e;
    o.x = o.x * f + v.x * e;
    o.y = o.y * f + v.y * e;
    o.z = o.z * f + v.z * e;
    o.w = o.w * f + v.w * e;
  }
};

// Parts of row r (of the sequence's rows) of key head `head` under one plan; true if there is one that covers all keys.
__device__ __forceinline__ bool join_parts(const CachedArgs& a, const CachedWork& w, int s, int head, int r, const float* whole, int lane,
                                           Joined& j) {
  int start;
  const int tiles = tiles_of(sequence(a, s, start));
  if (tiles == 0) return false;
  const CachedHeader h = *w.head;
  const int rows = a.rows_of_block, block = r / rows;
  const int64_t begin = w.base[s] + static_cast<int64_t>(block * a.hkv + head) * tiles;
  const int64_t first = stream_of(begin, h), last = stream_of(begin + tiles - 1, h);
  if (first == last) {
    if (a.partial) j.add(whole, lane);
    return true;
  }
#pragma unroll 4
  for (int64_t i = first; i <= last; ++i)
    j.add(w.slots + ((2 * i + (begin > range_begin(i, h) ? 1 : 0)) * rows + (r - block * rows)) * kPart, lane);
  return false;
}

__global__ void __launch_bounds__(128) cached_join_kernel(const CachedArgs a, const CachedWork w, const CachedArgs pa, const CachedWork pw) {
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (i >= static_cast<int64_t>(a.n) * a.t * a.hq) return;
  const int64_t token = i / a.hq;
  const int qh = static_cast<int>(i - token * a.hq), head = qh / a.group, in_group = qh - head * a.group;
  const int s = static_cast<int>(token / a.t), t = static_cast<int>(token - static_cast<int64_t>(s) * a.t);
  Joined j;
  if (a.partial) join_parts(pa, pw, 0, head, static_cast<int>(token) * a.group + in_group, pw.whole + i * kPart, lane, j);
  if (join_parts(a, w, s, head, t * a.group + in_group, w.whole + i * kPart, lane, j) && !a.partial) return;
  const bool some = j.l > 0.0f || j.l != j.l;
  const float inv = some ? 1.0f / j.l : 0.0f;
  *reinterpret_cast<uint2*>(a.O + token * a.ld_o + static_cast<int64_t>(qh) * 128 + 4 * lane) =
      make_uint2(pack_bf16x2(j.o.x * inv, j.o.y * inv), pack_bf16x2(j.o.z * inv, j.o.w * inv));
  if (lane == 0 && a.lse) a.lse[i] = some ? (j.m + log2f(j.l)) * 0.69314718055994531f : -INFINITY;
}

// ---- workspace

__host__ int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

struct Region {
  int64_t head, base, slots, whole, total;
};
// of one plan, from `at` on
__host__ Region region(int64_t at, int64_t n, int share, int rows_of_block, int64_t whole_rows) {
  Region r;
  r.head = at;
  r.base = up256(r.head + static_cast<int64_t>(sizeof(CachedHeader)));
  r.slots = up256(r.base + n * 8);
  r.whole = up256(r.slots + int64_t(2) * kSms * (kWarps / share) * rows_of_block * kPart * 4);
  r.total = up256(r.whole + whole_rows * kPart * 4);
  return r;
}
CachedWork work_at(void* ws, const Region& r) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  CachedWork w;
  w.head = reinterpret_cast<CachedHeader*>(p + r.head);
  w.base = reinterpret_cast<int64_t*>(p + r.base);
  w.slots = reinterpret_cast<float*>(p + r.slots);
  w.whole = reinterpret_cast<float*>(p + r.whole);
  return w;
}

// Warps that share tiles: as few as hold the rows, 8 or 16 each.
void shape_of(int64_t rows, int* nt, int* share) {
  *nt = rows <= 8 ? 1 : 2;
  *share = 1;
  while (*share < kWarps && *share * 16 < rows) *share *= 2;
}

Region own_region(const CachedArgs& a) {
  return region(0, a.n, a.share, a.rows_of_block, a.partial ? int64_t(a.n) * a.t * a.hq : 0);
}
Region prefix_region(const CachedArgs& a, const CachedArgs& p) {
  return region(own_region(a).total, 1, p.share, p.rows_of_block, int64_t(a.n) * a.t * a.hq);
}

}  // namespace

void cached_shape(CachedArgs* a) {
  int nt;
  shape_of(int64_t(a->t) * a->group, &nt, &a->share);
  a->rows_of_block = 8 * nt * a->share;
  a->blocks = static_cast<int32_t>((int64_t(a->t) * a->group + a->rows_of_block - 1) / a->rows_of_block);
}

int64_t cached_scratch_bytes(const CachedArgs& a, const CachedArgs* prefix) {
  return prefix ? prefix_region(a, *prefix).total : own_region(a).total;
}

cudaError_t launch_cached_attention(const CUtensorMap& k, const CUtensorMap& v, const CachedArgs& a, const CachedArgs* of, void* ws,
                                    int sms, cudaStream_t st) {
  static std::atomic<bool> ready_of[kMaxDevices];  // the shared-memory opt-in, per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!ready_of[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(cached_attention_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(cached_attention_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    ready_of[dev].store(true, std::memory_order_release);
  }
  const CachedWork w = work_at(ws, of ? prefix_region(*of, a) : own_region(a));
  const dim3 grid(static_cast<unsigned>(sms < kSms ? sms : kSms));
  return a.rows_of_block == 8 * a.share ? launch_pdl(cached_attention_kernel<1>, grid, dim3(kThreads), kSmem, 1, st, k, v, a, w)
                                        : launch_pdl(cached_attention_kernel<2>, grid, dim3(kThreads), kSmem, 1, st, k, v, a, w);
}

cudaError_t launch_cached_join(const CachedArgs& a, const CachedArgs* prefix, void* ws, cudaStream_t st) {
  const int64_t rows = int64_t(a.n) * a.t * a.hq;
  const CachedWork w = work_at(ws, own_region(a)), pw = prefix ? work_at(ws, prefix_region(a, *prefix)) : w;
  return launch_pdl(cached_join_kernel, dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, 1, st, a, w, prefix ? *prefix : a, pw);
}

cudaError_t take_cached_error(int* code) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_cached_err, sizeof(int));
  if (e != cudaSuccess) return e;
  *code = v;
  if (v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_cached_err, &zero, sizeof(int));
  }
  return e;
}

}  // namespace dm
