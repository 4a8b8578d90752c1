// cached_attention.cu -- attention of the last few tokens of each sequence over the 8-bit cache (rotary.cu writes it), and over
// rows that all sequences share.
//
// Keys and values are E4M3 codes with one power of two for each row and head, so K = k8 2^a and V = v8 2^b.  The scores are
// products of the codes times 2^a; with t = scale log2(e) q k + b and a reference m near the maximum of t, a key weighs w = 2^(t - m),
// which is its softmax weight times its value's 2^b: O = sum w v8, and the denominator is sum w 2^-b.
//
// Both products are transposed: a tile of 128 keys is the tensor core's 128 rows (S^T = K Q^T), then the 128 elements are (O^T = V^T
// P^T), so that codes go from memory to the tensor core as they are and few queries make a narrow product.  The narrow operand is a
// sum of terms of 8 bits in columns of their own.  q, scaled by a power of two for each row so that its largest value lies in [2^7,
// 2^8), is x1 + x2 / 16 in E4M3, x1 rounded and x2 the rest: exact down to 2^-14 of the largest, off by at most 2^-21 of it below.
// w is y1 + y2 / 8 + y3 / 32 in E5M2, three bits of fp16's eleven each: good to 2^-8, as bf16 would be, down to 2^-13, and to 2^-21.8
// below, 2^-30.8 of the row's largest weight.  (A key with most of the weight may stand before very many with 2^-20 of it each, which
// count together: two E4M3 terms, good to 2^-18 of the largest, lost 262143 keys 13 nats below the first, 8 % of O.)
// (With mma.sync, 8 rows a warp, codes have to be converted to f16, 3 - 4 clocks for two: one sequence of 262001 keys and 8 heads
// 130 us; its E4M3 form converts them too, 175.)
//
// A row is a token and one of the `group` query heads of a key head; R of them make 2 R columns of scores, for each 8 rows the first
// terms, then the second, and 3 R of O, for each 16 rows (or the only 8) one term after the other.  Warps of a block: one loads K and
// V by TMA into a ring, one issues the products, and four for each 16 rows hold the 128 keys (then elements), one a thread, which TMEM
// lane by lane suits: no sums across threads but at an item's end.  (What an item needs once is kept short: instructions that run once
// come from memory each time.)
//
// The tiles of all sequences, laid end to end, are cut into equal ranges, one for each group of `abreast` blocks, which take
// neighbouring key heads and so read a row's heads at about the same time.  What covers all keys of a row is written out; parts leave
// their m, denominator and O in the workspace, and a second kernel joins them in order.
// Bound: memory, 2 x 129 bytes a key and key head.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <climits>

#include "actfn.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace dm {

namespace {

__device__ int g_cached_err;

constexpr int kKeys = kCachedKeys;                 // of a tile
constexpr uint32_t kTile = kKeys * 128;            // bytes of K or V
constexpr int kSms = 152;                          // SMs that the workspace is sized for, at most
constexpr int kMaxAbreast = 8;
constexpr int kPart = 132;                         // floats of a partial row: 128 of O, m, denominator, two unused
constexpr int kJoinWarps = 8;
constexpr uint64_t kDrainNs = 200000000ull;

constexpr int kBlocks = 2;  // of an SM
constexpr int kErrSite = 0x26 << 4;  // of the waits, in the device error word
constexpr uint32_t kAbortAt = 260;  // in the control block

// For R rows: slots of the ring (a tile of K or of V each), columns of TMEM (two buffers of scores, O).
template <int R>
struct Shape {
  static constexpr int kRows = R < 16 ? R : 16, kGroups = R / kRows;  // groups of 128 threads that hold keys, and the rows of each
  static constexpr int kThreads = 64 + 128 * kGroups;                 // warps: 0 loads, 1 issues, from 2 on keys
  static constexpr uint32_t kSlots = R < 32 ? 5 : 4;                  // (six for 8 rows: 64 sequences of up to 8000 keys 91.6 us, five 88.4)
  static constexpr uint32_t kCols = 2 * R, kTerms = kRows;            // columns of scores; of one term of a group's O
  static constexpr uint32_t kOutCols = R == 8 ? 32 : 3 * R;           // of O (a product has a multiple of 16: 8 unused)
  static constexpr uint32_t kTmem = R == 8 ? 64 : R == 16 ? 128 : 256;
  static constexpr uint32_t kOperand = kCols * 128, kWeights = kOutCols * 128;  // bytes of Q and of P, two buffers each
  static constexpr uint32_t kCtrl = 4096;                                       // control block
  static constexpr int kSmem = 1024 + static_cast<int>(kCtrl + kSlots * kTile + 2 * kOperand + 2 * kWeights);
  static_assert(kBlocks * (kSmem + 1024 + 512) <= 233472 && 2 * kCols + kOutCols <= kTmem && kBlocks * kTmem <= 512, "memory of an SM");
};
// Weights are 2^kRaise where t is the maximum that m was taken from; the maximum may rise by kBehind (in base 2) before O and the
// denominator are brought to a new m, so that they stay below E5M2's 57344 = 2^15.807.  (With less to rise m moves more often, at 1 us a
// time: 48 sequences behind 16001 shared rows 66.2 us with 4.8, 63.1 so; with a lower start more of the small weights is lost.)
constexpr float kRaise = 9.0f, kBehind = 6.75f;
constexpr float kTerm = 0.0625f;                      // of q's second terms
constexpr float kSecond = 0.125f, kThird = 0.03125f;  // of the weights' terms

// ---- work: tiles of all items (sequence, block of rows, `abreast` key heads) in order.  What an item costs beside its tiles counts as
// kItem of them, before its first: units.  (256 tokens over up to 1000 keys of one head 22.7 us without, 19.4 so, 18.5 with two; 48 sequences
// behind 16001 shared rows 71.8, 63.1, 65.0.)
constexpr int kItem = 1;

struct CachedHeader {
  int64_t units;       // of all items
  int64_t each;        // of a range; the first `rest` ranges have one more
  int32_t rest, ranges;
};

struct CachedWork {
  CachedHeader* head;
  int64_t* base;    // units before each sequence
  float* slots;     // two for each range, of R partial rows for each head abreast
  float* whole;     // partial rows of items that were not cut, by token and head (with a shared prefix)
};

// The list of work: the rows that all sequences share, where there are some (entry 0, whose rows are all tokens'), then the sequences.
__device__ __forceinline__ bool is_shared(const CachedArgs& a, int s) { return s < a.shared; }
__device__ __forceinline__ int rows_of(const CachedArgs& a, int s) { return is_shared(a, s) ? a.shared_rows : a.rows; }
__device__ __forceinline__ int blocks_of(const CachedArgs& a, int s) { return is_shared(a, s) ? a.shared_blocks : a.blocks; }
__device__ __forceinline__ int64_t first_token(const CachedArgs& a, int s) {
  return is_shared(a, s) ? 0 : static_cast<int64_t>(s - a.shared) * a.t;
}

// First row and length of an entry; one whose rows leave the cache gets none and is recorded.
__device__ __forceinline__ void given_rows(const CachedArgs& a, int s, int& start, int& len) {
  start = is_shared(a, s) ? a.prefix[0] : a.k_start[s - a.shared];
  len = is_shared(a, s) ? a.prefix[1] : a.k_len[s - a.shared];
}
__device__ __forceinline__ int checked(const CachedArgs& a, int& start, int len) {
  if (start < 0 || len < 0 || len > a.cache_rows || start > a.cache_rows - len) {
    atomicCAS(&g_cached_err, 0, kPackedBadLengths);
    start = len = 0;
  }
  return len;
}
__device__ __forceinline__ int sequence(const CachedArgs& a, int s, int& start) {
  int len;
  given_rows(a, s, start, len);
  return checked(a, start, len);
}
__device__ __forceinline__ int tiles_of(int len) { return (len + kKeys - 1) / kKeys; }
__device__ __forceinline__ int units_of(int tiles) { return tiles > 0 ? tiles + kItem : 0; }

__device__ __forceinline__ int64_t divide(int64_t x, int64_t y) {  // x, y >= 0; nearly always within 32 bits
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}
// Where range i begins, and the range that unit x belongs to.
__device__ __forceinline__ int64_t range_begin(int64_t i, const CachedHeader& h) { return i * h.each + (i < h.rest ? i : h.rest); }
__device__ __forceinline__ int64_t range_of(int64_t x, const CachedHeader& h) {
  const int64_t longer = h.rest * (h.each + 1);
  return x < longer ? divide(x, h.each + 1) : h.rest + divide(x - longer, h.each);
}

// An item's part in a range: keys of tiles t0 .. t1 - 1 of entry s.
struct Piece {
  int s, start, len, tiles;
  int block, head;  // block of rows, first of the key heads abreast
  int t0, t1;
  int64_t at;       // the item's first unit
};

// Sets t1; false where there is none (past the range, or, where lengths change while the kernel reads them, past the sequences).
__device__ __forceinline__ bool close_piece(const CachedArgs& a, Piece& p, int64_t hi) {
  const int64_t left = hi - p.at - kItem;
  p.t1 = p.tiles < left ? p.tiles : static_cast<int>(left);
  return p.t1 > p.t0 && p.s < a.n + a.shared;
}
// (next_start, next_len: those of the entry behind p's, loaded by the call before, so that none waits for them.)
__device__ __forceinline__ bool next_piece(const CachedArgs& a, Piece& p, int64_t hi, int& next_start, int& next_len) {
  p.at += units_of(p.tiles);
  p.t0 = 0;
  p.head += a.abreast;
  if (p.head >= a.hkv) {
    p.head = 0;
    if (++p.block >= blocks_of(a, p.s)) {
      p.block = 0;
      const int entries = a.n + a.shared;
      do {
        ++p.s;
        p.start = next_start;
        p.len = p.s < entries && p.at < hi ? checked(a, p.start, next_len) : 0;
        p.tiles = tiles_of(p.len);
        if (p.s + 1 < entries) given_rows(a, p.s + 1, next_start, next_len);
      } while (p.tiles == 0 && p.s < entries && p.at < hi);
    }
  }
  return close_piece(a, p, hi);
}

// ---- instructions

// D[tmem] (+)= A . B^T, operands of 8 bits in shared memory, fp32 accumulator, 32 of the reduction.
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
constexpr uint32_t kE5m2Columns = 1u << 10;  // of the instruction's descriptor: B's format
// Descriptor of an operand without swizzle whose rows along the reduction are pieces of 16 bytes (16 columns), one after the other; the
// next 16 columns `stride` bytes further.  (8 rows of 16 bytes are a unit; bits 16 - 29: the distance of units along the reduction, bits
// 32 - 45: along the columns.)
__device__ __forceinline__ uint64_t sdesc_pieces(uint32_t saddr, uint32_t stride) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(128u >> 4) << 16 |
         static_cast<uint64_t>((stride & 0x3FFFFu) >> 4) << 32 | static_cast<uint64_t>(1) << 46;
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
// A tile of codes to shared memory, the first to leave L2 again: they are read once, or by blocks that run at about the same time (64
// sequences of up to 8000 keys 88.4 us, 92.2 without).
__device__ __forceinline__ uint64_t read_once_policy() {
  uint64_t policy;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t head, int32_t row, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(head), "r"(row), "l"(policy)
      : "memory");
}
// The threads that hold a group's keys meet.
__device__ __forceinline__ void group_sync(int group) { asm volatile("bar.sync %0, 128;" ::"r"(group + 1) : "memory"); }
__device__ __forceinline__ bool group_any(int group, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "bar.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(group + 1), "r"(static_cast<uint32_t>(x))
      : "memory");
  return r != 0;
}

// Whether the phase has completed, without any wait.
__device__ __forceinline__ bool arrived(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// mbar_wait with all but its first look out of the way: the loop over tiles is long as it is, and instructions that it passes over cost
// it their fetching and the registers of their arguments.  (The barriers lie at the start of the control block, which is aligned to 1024 bytes.)
__device__ __noinline__ bool arrival_awaited(uint32_t bar, uint32_t parity, int site) {
  volatile int* abort_flag = static_cast<volatile int*>(__cvta_shared_to_generic((bar & ~1023u) + kAbortAt));
  return mbar_wait(bar, parity, abort_flag, &g_cached_err, kErrSite + site);
}
__device__ __forceinline__ bool arrival(uint32_t bar, uint32_t parity, int site) {
  return mbar_try_wait(bar, parity) || arrival_awaited(bar, parity, site);
}

__device__ __forceinline__ uint16_t e4m3_of_f16(__half2 x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(*reinterpret_cast<const uint32_t*>(&x)));
  return r;
}
__device__ __forceinline__ __half2 f16_of_e4m3(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return *reinterpret_cast<const __half2*>(&r);
}
// The two terms of x and y (at most 448 in size; f16 holds 3 bits more than the terms do).
__device__ __forceinline__ void two_terms(float x, float y, uint32_t& first, uint32_t& second) {
  const __half2 v = __floats2half2_rn(x, y);
  const uint16_t f = e4m3_of_f16(v);
  first = f;
  second = e4m3_of_f16(__hmul2(__hsub2(v, f16_of_e4m3(f)), __float2half2_rn(16.0f)));
}
// The three terms of weights x and y (at most 2^15.75; fp16's upper byte is the E5M2 value next to zero): the first two in the upper
// bytes of the halves, the third, rounded, in two bytes.  All but the two roundings is exact.  NaN stays in the first.
__device__ __forceinline__ void three_terms(float x, float y, uint32_t& first, uint32_t& second, uint16_t& third) {
  auto upper = [](uint32_t v) {
    v &= 0xFF00FF00u;
    return *reinterpret_cast<const __half2*>(&v);
  };
  const __half2 v = __floats2half2_rn(x, y);
  first = *reinterpret_cast<const uint32_t*>(&v);
  const __half2 rest = __hmul2(__hsub2(v, upper(first)), __float2half2_rn(8.0f));
  second = *reinterpret_cast<const uint32_t*>(&rest);
  const __half2 last = __hmul2(__hsub2(rest, upper(second)), __float2half2_rn(4.0f));
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(third) : "r"(*reinterpret_cast<const uint32_t*>(&last)));
}
__device__ __forceinline__ uint32_t upper_bytes(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7531); }
// A byte of a list that is read on from there: memory brings 128 bytes at a time to L2, not 32.
__device__ __forceinline__ int load_line(const uint8_t* p) {
  uint32_t x;
  asm volatile("ld.global.L2::128B.u8 %0, [%1];" : "=r"(x) : "l"(p));
  return static_cast<int>(x);
}

// A row of an item, in shared memory
struct __align__(16) Row {
  float scale;   // of the scores of its q, in base 2
  float base;    // m (0 while there is none)
  int limit;     // keys that it sees
  int begun;     // whether there is an m
};

// ... and, at the item's end, where its results go
struct __align__(16) OutRow {
  int64_t at;    // of O, the partial results or the whole ones
  float factor;
  int limit;
};

enum : int { B_FULL = 0, B_EMPTY = 8, B_Q_FULL = 16, B_S_FULL = 18, B_P_FULL = 20, B_PV_DONE = 22, B_DRAIN = 24, B_EXPS = 25,
             B_Q_EMPTY = 29, B_READY = 31, B_COUNT = 32 };
// Control block: barriers, then 256: TMEM address, abort flag, flags of warps; 512: pieces (two items', the range's first); 1024: rows of two items; 2048: four warps'
// maxima or sums of 32 rows; 2560: by how much m moved, and the factor for what was added up before; then the exponents of four tiles' keys
constexpr uint32_t kFlagsAt = 288, kPiecesAt = 512, kRowsAt = 1024, kSumsAt = 2048, kMovesAt = 2560, kExpsAt = kMovesAt + 512;
constexpr uint32_t kExpTiles = 4;
static_assert(sizeof(Piece) * 3 <= kRowsAt - kPiecesAt && 8 * B_COUNT <= 256, "control block");

// An item's rows to shared memory, in two terms, by warps whose lanes take 16 a row: this one rows first, first + step, ...  Rows 16 c + n
// (first terms) and 16 c + 8 + n (second) of the product's narrow operand are row 8 c + n of the item, 128 bytes each under the
// 128-byte swizzle.
__device__ __noinline__ void prepare_rows(const CachedArgs& a, int s, int len, int head, int r0, uint32_t to, Row* rows, int lane,
                                          int first, int step) {
  const int piece = lane & 15, all = rows_of(a, s), top = (min(a.rows_of_block, all - r0) + 7) & ~7;
#pragma unroll 1
  for (first += lane >> 4; first - (lane >> 4) < top; first += 4 * step) {
    uint4 u[4];
    float amax[4];
    int token[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + first + step * i;
      u[i] = make_uint4(0u, 0u, 0u, 0u);
      token[i] = static_cast<int>(static_cast<uint32_t>(r) / static_cast<uint32_t>(a.group));
      if (first + step * i < top && r < all) {
        const uint16_t* q =
            a.Q + (first_token(a, s) + token[i]) * a.ld_q + (static_cast<int64_t>(head) * a.group + r - token[i] * a.group) * 128;
        u[i] = reinterpret_cast<const uint4*>(q)[piece];
      }
    }
    auto value = [&](int i, int e) {
      const uint32_t x = e < 2 ? u[i].x : e < 4 ? u[i].y : e < 6 ? u[i].z : u[i].w;
      return e & 1 ? bf16hi(x) : bf16lo(x);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      amax[i] = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) amax[i] = fmaxf(amax[i], fabsf(value(i, e)));
    }
#pragma unroll
    for (int o = 1; o < 16; o <<= 1)
#pragma unroll
      for (int i = 0; i < 4; ++i) amax[i] = fmaxf(amax[i], __shfl_xor_sync(0xFFFFFFFFu, amax[i], o));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int in = first + step * i, c = in >> 3, n = in & 7;
      // 2^up brings the largest into [2^7, 2^8) (an infinity becomes NaN, as its scores would)
      const int up = amax[i] > 0.0f && amax[i] < INFINITY ? min(7 + 127 - static_cast<int>(__float_as_uint(amax[i]) >> 23), 120) : 0;
      const float f = amax[i] < INFINITY ? __int_as_float((up + 127) << 23) : NAN;
      uint32_t one[4], two[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) two_terms(value(i, 2 * e) * f, value(i, 2 * e + 1) * f, one[e], two[e]);
      if (in < top) {
        const uint32_t at = to + static_cast<uint32_t>(c * 2048 + n * 128 + (((piece >> 1) ^ n) << 4) + (piece & 1) * 8);
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(one[0] | one[1] << 16), "r"(one[2] | one[3] << 16) : "memory");
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at + 1024u), "r"(two[0] | two[1] << 16), "r"(two[2] | two[3] << 16) : "memory");
        if (piece == 0) {
          const int limit = r0 + in >= all ? 0 : is_shared(a, s) ? len : len - a.t + token[i] + 1;
          rows[in] = {a.scale_log2 * __int_as_float((127 - up) << 23), 0.0f, limit, 0};
        }
      }
    }
  }
  fence_proxy_async_smem();
}

// Whether the threads that hold the keys prepare an item's rows (the range's first they always do).  The loading warp takes 2.5 us for
// eight, while the others work on the item before, but ten for 32: 16 sequences of up to 3001 keys, 35 rows each for 4 heads 32.0 us if it
// prepares all, 28.8 so.
template <int R>
__device__ __forceinline__ bool keys_prepare(const CachedArgs& a, const Piece& p) {
  return R > 8 && rows_of(a, p.s) - p.block * R > 8;
}

// Sums over the warp of each of ROWS values: lane i gets that of row i / (32 / ROWS).
template <int ROWS>
__device__ __forceinline__ float row_sums(float (&v)[ROWS], int lane) {
  int o = 16;
#pragma unroll
  for (int half = ROWS / 2; half > 0; half >>= 1, o >>= 1) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = upper ? v[i + half] : v[i], give = upper ? v[i] : v[i + half];
      v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
    }
  }
  float sum = v[0];
  for (; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  return sum;
}

template <int R>
__global__ void __launch_bounds__(Shape<R>::kThreads, kBlocks)
    cached_attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                            const __grid_constant__ CachedArgs a, const CachedWork w) {
  using S = Shape<R>;
  constexpr uint32_t kSlots = S::kSlots;
  constexpr int kThreads = S::kThreads, kRows = S::kRows, kChunks = kRows / 8;  // rows and chunks of 8 of a group
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + (((smem_u32(smem_raw) + 1023u) & ~1023u) - smem_u32(smem_raw));
  __shared__ int64_t warp_sums[kThreads / 32];
  const uint32_t bar0 = smem_u32(smem), ring = bar0 + S::kCtrl, q_at = ring + kSlots * kTile, p_at = q_at + 2 * S::kOperand;
  auto bar = [bar0](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + 256);
  Piece* pieces = reinterpret_cast<Piece*>(smem + kPiecesAt);
  Row* all_rows = reinterpret_cast<Row*>(smem + kRowsAt);
  float* sums = reinterpret_cast<float*>(smem + kSumsAt);
  float2* moves = reinterpret_cast<float2*>(smem + kMovesAt);
  volatile uint32_t* flags_of = reinterpret_cast<volatile uint32_t*>(smem + kFlagsAt);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i)
      mbar_init(bar(i), i == B_P_FULL || i == B_P_FULL + 1 || i == B_READY ? 4 * S::kGroups : i >= B_Q_EMPTY ? 4 * S::kGroups + 1
                        : i >= B_EXPS || i == B_Q_FULL || i == B_Q_FULL + 1 ? 32 : 1);
    *reinterpret_cast<volatile int*>(smem + kAbortAt) = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), S::kTmem);
    tmem_relinquish();
  }
  pdl_launch();
  pdl_wait();

  // ---- the plan, by every block for itself: tiles (times blocks of rows) before each thread's entries
  const int entries = a.n + a.shared, subs = a.hkv / a.abreast;
  const int per = (entries + kThreads - 1) / kThreads, s0 = min(static_cast<int>(threadIdx.x) * per, entries), s1 = min(s0 + per, entries);
  int64_t mine = 0;
  int start0 = 0, len0 = 0;  // of the thread's last entry
  for (int s = s0; s < s1; ++s) {
    len0 = sequence(a, s, start0);
    mine += static_cast<int64_t>(units_of(tiles_of(len0))) * blocks_of(a, s);
  }
  int64_t sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) warp_sums[warp] = sum;
  if (threadIdx.x == 0) pieces[2] = Piece{};
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int64_t total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i == warp) sum += total;
    total += warp_sums[i];
  }
  CachedHeader h;
  h.units = total * subs;
  {
    const int most = static_cast<int>(gridDim.x) / a.abreast;
    h.ranges = h.units < most ? (h.units > 0 ? static_cast<int>(h.units) : 1) : most;
    h.each = divide(h.units, h.ranges);
    h.rest = static_cast<int>(h.units - h.each * h.ranges);
  }
  const int lane_head = blockIdx.x % a.abreast;  // of the heads abreast
  const int64_t range = blockIdx.x / a.abreast;
  const bool work = h.units > 0 && range < h.ranges;
  const int64_t lo = work ? range_begin(range, h) : 0, hi = work ? range_begin(range + 1, h) : 0;
  // the range's first piece: unit lo is unit lo - done of entry p.s
  auto enter = [&](Piece p, int64_t done) {
    const int units = units_of(p.tiles), item = static_cast<int>(divide(lo - done, units));
    p.at = done + static_cast<int64_t>(item) * units;
    p.block = item / subs;
    p.head = (item - p.block * subs) * a.abreast;
    p.t0 = max(static_cast<int>(lo - p.at) - kItem, 0);
    if (close_piece(a, p, hi)) pieces[2] = p;
  };
  const int64_t mine_at = (sum - mine) * subs;
  if (work && mine_at <= lo && lo < mine_at + mine * subs) {
    // one thread has it; with several entries a thread it passes over those before
    Piece p = {};
    p.s = s0;
    int64_t done = mine_at;
    p.start = start0;
    p.len = len0;
    for (;; ++p.s) {
      if (per > 1) p.len = p.s < s1 ? sequence(a, p.s, p.start) : 0;
      p.tiles = tiles_of(p.len);
      const int64_t all = static_cast<int64_t>(units_of(p.tiles)) * blocks_of(a, p.s) * subs;
      if (lo < done + all || p.s >= s1) break;
      done += all;
    }
    if (p.tiles > 0) enter(p, done);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *w.head = h;
  if (threadIdx.x % gridDim.x == blockIdx.x) {  // for the second kernel
    int64_t at = mine_at;
    for (int s = s0; s < s1; ++s) {
      int start;
      w.base[s] = at;
      at += static_cast<int64_t>(units_of(tiles_of(sequence(a, s, start)))) * blocks_of(a, s) * subs;
    }
  }
  __syncthreads();

  if (work && warp == 0) {
    // ---------------- loads: K and V of one tile after the other, and its keys' exponents, which the lanes ask for (four keys each)
    // before they wait for the tile's places, and store before the next tile.  (Loaded by the threads that use them, a tile ahead, they were waited for:
    // 64 sequences of up to 8000 keys 101 us.)  Four tiles of them are kept: V of the third tile before is read by then.
    // It also prepares each item but the first: its piece and (few) rows for the others, two items at a time.
    Piece p = pieces[2];
    uint32_t slot = 0, round = 0, made = 0, item = 0;
    const bool one = elect_one();
    bool ok = true, more = p.t1 > p.t0;
    const uint64_t policy = read_once_policy();
    int next_start = 0, next_len = 0;
    if (p.s + 1 < entries) given_rows(a, p.s + 1, next_start, next_len);
    int of_keys[4], of_values[4];  // (joined where they are stored, so that nothing waits for them before)
    auto store = [&] {  // those of tile made - 1
      const uint32_t to = bar0 + kExpsAt + ((made - 1) & (kExpTiles - 1)) * (2u * kKeys) + 2u * lane;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        asm volatile("st.shared.u16 [%0], %1;" ::"r"(to + 64u * i), "h"(static_cast<unsigned short>(of_keys[i] | of_values[i] << 8)) : "memory");
      mbar_arrive(bar(B_EXPS + ((made - 1) & (kExpTiles - 1))));
    };
    auto wait = [&](int b, uint32_t parity, int site) {  // the same in the whole warp
      ok = __all_sync(0xFFFFFFFFu, ok && arrival(bar(b), parity & 1u, site));
    };
    for (;; ++item) {
      for (int tile = p.t0; tile <= p.t1; ++tile) {
        if (tile < p.t1) {
          if (made > 0 && ok) store();
          const int row = p.start + tile * kKeys;
          const int64_t list = (p.head + lane_head) * a.ld_exp + row;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int in = 32 * i + lane;
            of_keys[i] = of_values[i] = 127;  // (what lies past the keys may be anything)
            if (tile * kKeys + in < p.len) {
              of_keys[i] = load_line(a.k_exp + list + in);
              of_values[i] = load_line(a.v_exp + list + in);
            }
          }
#pragma unroll
          for (int value = 0; value < 2; ++value) {
            if (round > 0) wait(B_EMPTY + slot, round - 1, 1);
            if (ok && one) {
              mbar_arrive_expect_tx(bar(B_FULL + slot), kTile);
              load_tile(ring + slot * kTile, value ? &map_v : &map_k, bar(B_FULL + slot), p.head + lane_head, row, policy);
            }
            if (++slot == kSlots) {
              slot = 0;
              ++round;
            }
          }
          ++made;
        }
        if (tile == p.t0 && item > 0) {  // (or there is no item, and the others learn it)
          if (item >= 2) wait(B_Q_EMPTY + (item & 1u), (item >> 1) + 1, 12);
          if (lane == 0) pieces[item & 1u] = p;
          if (more && !keys_prepare<R>(a, p))
            prepare_rows(a, p.s, p.len, p.head + lane_head, p.block * R, q_at + (item & 1u) * S::kOperand, all_rows + (item & 1u) * R, lane, 0, 2);
          mbar_arrive(bar(B_Q_FULL + (item & 1u)));
        }
        if (!ok || !more) break;
      }
      if (!ok || !more) break;
      more = next_piece(a, p, hi, next_start, next_len);
      if (!more) p.t1 = p.t0;
    }
    if (made > 0 && ok) store();
    if (!ok) {  // copies in flight land before the block leaves
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 100000ull) {
      }
    }
  } else if (work && warp == 1) {
    // ---------------- products: S of a tile while the one before it is weighed, then O += V^T P of that
    const bool one = elect_one();
    const uint64_t ring_desc = sdesc_sw128(ring, 16, 1024);
    bool ok = true;
    auto wait = [&](int b, uint32_t parity, int site) {  // the same in the whole warp
      ok = __all_sync(0xFFFFFFFFu, ok && arrival(bar(b), parity & 1u, site));
    };
    int tile = 0, tile0 = 0, tile1 = 0;
    bool more = false;
    uint32_t item = 0, made = 0, slot_k = 0, round_k = 0, slot_v = 1, round_v = 0, item_columns = 0, readied = 0;
    auto enter = [&] {  // item `item`
      wait(B_Q_FULL + (item & 1u), item >> 1, 2);
      const Piece& p = pieces[item & 1u];
      tile = tile0 = p.t0;
      tile1 = p.t1;
      item_columns = 16u * static_cast<uint32_t>((min(R, rows_of(a, p.s) - p.block * R) + 7) >> 3);
      more = ok && tile1 > tile0;
      if (more && item > 0 && keys_prepare<R>(a, p)) wait(B_READY, readied++, 14);
    };
    auto next_ready = [&] {  // whether there is no more to wait for before the next item (what the keys' threads prepare comes after its turn)
      const uint32_t next = item + 1;
      return __all_sync(0xFFFFFFFFu, arrived(bar(B_Q_FULL + (next & 1u)), (next >> 1) & 1u) && !keys_prepare<R>(a, pieces[next & 1u]));
    };
    uint32_t columns = 0, columns_before = 0;  // of the last tile and of the one before it; bit 31: the item's first
    auto advance = [](uint32_t& slot, uint32_t& round) {
      slot += 2;
      if (slot >= kSlots) {
        slot -= kSlots;
        ++round;
      }
    };
    auto scores = [&] {
      wait(B_FULL + slot_k, round_k, 3);
      columns_before = columns;
      columns = item_columns;
      tc_fence_after();
      if (ok && one) {
        const uint32_t id = idesc_e4m3_f32(128, static_cast<int>(columns), false, false);
        const uint64_t dk = ring_desc + ((slot_k * kTile) >> 4), dq = sdesc_sw128(q_at + (item & 1u) * S::kOperand, 16, 1024);
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) umma_f8(tmem + (made & 1u) * S::kCols, dk + 2 * k, dq + 2 * k, id, k != 0);
        umma_commit(bar(B_S_FULL + (made & 1u)));
        umma_commit(bar(B_EMPTY + slot_k));
        if (tile + 1 == tile1) umma_commit(bar(B_Q_EMPTY + (item & 1u)));
      }
      __syncwarp();
      if (tile == tile0) columns |= 1u << 31;
      advance(slot_k, round_k);
      ++made;
      ++tile;
    };
    enter();
    if (more) scores();
    for (uint32_t j = 0; j < made && ok; ++j) {
      bool last = tile == tile1;  // of its item
      if (last && next_ready()) {
        ++item;
        enter();
        last = false;
      }
      const bool ahead = !last && more;
      if (ahead) scores();
      const uint32_t mine = ahead ? columns_before : columns;
      wait(B_P_FULL + (j & 1u), j >> 1, 4);
      wait(B_FULL + slot_v, round_v, 5);
      tc_fence_after();
      if (ok && one) {
        // (groups of 16 rows; scores have 16 columns for 8)
        const uint32_t out_columns = S::kGroups > 1 && (mine & 0xFFFFu) <= 32 ? S::kOutCols / S::kGroups : S::kOutCols;
        const uint32_t id = idesc_e4m3_f32(128, static_cast<int>(out_columns), true, true) | kE5m2Columns;
        const uint64_t dv = ring_desc + ((slot_v * kTile) >> 4), dp = sdesc_pieces(p_at + (j & 1u) * S::kWeights, kKeys * 16);
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k)
          umma_f8(tmem + 2 * S::kCols, dv + k * (4096u >> 4), dp + k * (512u >> 4), id, !(mine >> 31 && k == 0));
        umma_commit(bar(B_PV_DONE + (j & 1u)));
        umma_commit(bar(B_EMPTY + slot_v));
      }
      __syncwarp();
      advance(slot_v, round_v);
      if (last) {  // (the next item's rows may have to wait for what the last product goes to)
        ++item;
        enter();
        if (more) scores();
      }
    }
    if (one) umma_commit(bar(B_DRAIN));
    __syncwarp();
    const uint64_t t0 = global_timer_ns();  // what was issued ends before the block frees its memory, whatever happened
    while (!mbar_try_wait(bar(B_DRAIN), 0) && global_timer_ns() - t0 < kDrainNs) {
    }
  } else if (work) {
    // ---------------- keys: a thread has one key of each tile, and one element of O, both the number of its TMEM lane, for its group's
    // rows.  After a wait that ran out these warps go on (every later one ends at once), so that they meet at their barriers, but write
    // nothing.
    const int group = (threadIdx.x - 64) >> 7, x = (threadIdx.x - 64) & 127, quarter = (warp & 3) * 32, me = quarter + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter) << 16) + static_cast<uint32_t>(group * 2 * kRows);
    const uint32_t out_lanes = lanes + 2 * S::kCols + static_cast<uint32_t>(group * kRows);  // (three terms of its rows, where scores have two)
    sums += group * 4 * kRows;
    moves += group * kRows;
    flags_of += group * 4;
    auto groups_sync = [&] {
      if (S::kGroups > 1) asm volatile("bar.sync %0, %1;" ::"n"(S::kGroups + 1), "n"(128 * S::kGroups) : "memory");
    };
    auto keys_any = [&](bool x) {
      uint32_t r;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\t"
          "setp.ne.b32 p, %3, 0;\n\t"
          "bar.red.or.pred q, %1, %2, p;\n\t"
          "selp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(r)
          : "n"(S::kGroups + 1), "n"(128 * S::kGroups), "r"(static_cast<uint32_t>(x))
          : "memory");
      return r != 0;
    };
    bool ok = true;
    auto wait = [&](int b, uint32_t parity, int site) {
      ok = arrival(bar(b), parity & 1u, site) && ok;
    };
    // the range's first item, by all
    {
      const Piece p = pieces[2];
      prepare_rows(a, p.s, p.len, p.head + lane_head, p.block * R, q_at, all_rows, lane, 2 * (warp - 2), 8 * S::kGroups);
      if (threadIdx.x == 64) pieces[0] = p;
    }
    keys_any(false);
    if (warp == 2) mbar_arrive(bar(B_Q_FULL));
    uint32_t readied = 0;
    uint32_t j = 0;  // tiles so far
    for (uint32_t item = 0;; ++item) {
      wait(B_Q_FULL + (item & 1u), item >> 1, 13);
      // (The rest of the piece is read again where it is needed: with two groups registers are short, and 48 sequences behind 16001 shared
      // rows took 62.5 us with more of them held, 59 so.)
      int tile, end, count, least;
      {
        const Piece p = pieces[item & 1u];
        if (keys_any(!ok) || p.t1 <= p.t0) break;  // (the same for all: nobody is left at a barrier)
        if (item > 0 && keys_prepare<R>(a, p)) {
          prepare_rows(a, p.s, p.len, p.head + lane_head, p.block * R, q_at + (item & 1u) * S::kOperand, all_rows + (item & 1u) * R, lane,
                       2 * (warp - 2), 8 * S::kGroups);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_READY));
          wait(B_READY, readied++, 14);
        }
        tile = p.t0;
        end = p.t1;
        count = min(kRows, rows_of(a, p.s) - p.block * R - group * kRows);
        least = is_shared(a, p.s) ? p.len : p.len - a.t + p.block * R / a.group + 1;  // keys that every row sees
      }
      const int chunks = (count + 7) >> 3;  // (none: below 0)
      Row* rows = all_rows + (item & 1u) * R + group * kRows;
      int nan_key = INT_MAX;  // the first key, of those that not all rows see, with NaN in this thread's element
      float l[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) l[r] = 0.0f;
      bool force = true;  // rows without an m

      for (bool first = true; tile < end; ++tile, ++j, first = false) {
        const int key0 = tile * kKeys;
        const bool tail = key0 + kKeys > least;
        wait(B_EXPS + (j & (kExpTiles - 1)), j / kExpTiles, 11);
        unsigned short packed;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(packed) : "r"(bar0 + kExpsAt + (j & (kExpTiles - 1)) * (2u * kKeys) + 2u * me) : "memory");
        const int exps = packed;
        const float key_scale = __int_as_float((exps & 255) << 23), bias = static_cast<float>((exps >> 8) - 127);
        float unbias = __int_as_float((254 - (exps >> 8)) << 23);
        const uint32_t from = lanes + (j & 1u) * S::kCols;
        wait(B_S_FULL + (j & 1u), j >> 1, 6);
        tc_fence_after();
        float d[kRows];  // t - m
        uint32_t flags = 0;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (c < chunks) {
            uint32_t y[16];
            tmem_ld16(from + 16u * c, y);
            tmem_ld_wait();
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float2 row = *reinterpret_cast<const float2*>(rows + 8 * c + i);
              const float z = fmaf(__uint_as_float(y[8 + i]), kTerm, __uint_as_float(y[i])) * key_scale;
              d[8 * c + i] = fmaf(z, row.x, bias - row.y);
            }
            if (__builtin_expect(tail, 0)) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                if (key0 + me >= rows[8 * c + i].limit) d[8 * c + i] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, d[8 * c + i]);
            flags |= static_cast<uint32_t>(top > kRaise + kBehind) << c;
          }
        }
        if (force) {
          flags = chunks > 0 ? (1u << chunks) - 1u : 0u;
        } else if (kChunks == 1) {
          flags = group_any(group, flags != 0) ? 1u : 0u;
        } else {
          flags = __reduce_or_sync(0xFFFFFFFFu, flags);
          // (in turn in two places: a warp may write the next tile's before another has read this one's)
          volatile uint32_t* of = flags_of + (j & 1u) * (4 * S::kGroups);
          if (lane == 0) of[warp & 3] = flags;
          group_sync(group);
          flags = (of[0] | of[1]) | (of[2] | of[3]);
        }
        if (__builtin_expect(flags != 0, 0)) {
          // A value of zeros adds nothing to O, so it may not set the m of those that do (the cache gives it 2^0, and values of size 0.05 have
          // 2^-11): its power of two counts as the least.  So does that of zeros and NaN, which is NaN with any weight.  (Looked at where m moves
          // alone, so that only items' first tiles wait for their values: 48 sequences behind 16001 shared rows 63.2 us, 61.4 without.)
          {
            const uint32_t slot_v = (2 * j + 1) % kSlots, v_at = ring + slot_v * kTile;
            wait(B_FULL + slot_v, (2 * j + 1) / kSlots, 15);
            if ((exps >> 8) > 127 - kCacheExpMax) {
              bool zeros = true;
              for (int i = 0; i < 8 && zeros; ++i) {
                const uint4 u = ld_shared_v4(v_at + static_cast<uint32_t>(me * 128 + ((i ^ (me & 7)) << 4)));
                auto some = [](uint32_t codes) { return ((codes & 0x7F7F7F7Fu) + 0x01010101u) & 0x7E7E7E7Eu; };  // but 0 and 0x7F
                zeros = ((some(u.x) | some(u.y)) | (some(u.z) | some(u.w))) == 0;
              }
              if (zeros) {
                const float less = bias + static_cast<float>(kCacheExpMax);
#pragma unroll
                for (int r = 0; r < kRows; ++r) d[r] -= less;
                unbias = static_cast<float>(1ull << kCacheExpMax);
              }
            }
          }
          // the rows' maxima.  Where one is well above m, m moves, and with it those of its eight rows that have risen at all: what costs is
          // the visit (1 us; when 4.8 were left to rise, 18 of 100 tiles of 48 rows over 16001 keys had one, and 64.5 us became 62.5), not the row.
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c < chunks && (flags >> c & 1u)) {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float z = d[8 * c + i];
                const int bits = __float_as_int(z == z ? z : -INFINITY);
                const int top = __reduce_max_sync(0xFFFFFFFFu, bits ^ ((bits >> 31) & 0x7FFFFFFF));  // (ordered as the floats are)
                if (lane == 0) sums[(warp & 3) * kRows + 8 * c + i] = __int_as_float(top ^ ((top >> 31) & 0x7FFFFFFF));
              }
            }
          group_sync(group);
          bool without = false;
          if (x < 8 * chunks && (flags >> (x >> 3) & 1u)) {
            const float top = fmaxf(fmaxf(sums[x], sums[kRows + x]), fmaxf(sums[2 * kRows + x], sums[3 * kRows + x]));
            Row row = rows[x];
            float2 move = make_float2(0.0f, 1.0f);
            if (row.begun ? top > kRaise : top > -INFINITY) {
              move = make_float2(top - kRaise, row.begun ? ex2_approx(kRaise - top) : 0.0f);
              row.base += move.x;
              row.begun = 1;
              rows[x] = row;
            }
            moves[x] = move;
            without = !row.begun && x < count;
          }
          force = group_any(group, without);
          if (!first) {
            wait(B_PV_DONE + ((j - 1) & 1u), (j - 1) >> 1, 7);
            tc_fence_after();
          }
#pragma unroll
          for (int r = 0; r < kRows; ++r)
            if (flags >> (r >> 3) & 1u) {
              const float2 move = moves[r];
              d[r] -= move.x;
              l[r] *= move.y;
            }
#pragma unroll 1
          for (int c = 0; c < chunks && !first; ++c)
            if (flags >> c & 1u) {
#pragma unroll 1
              for (uint32_t at = out_lanes + 8u * c; at < out_lanes + 3 * S::kTerms; at += S::kTerms) {
                uint32_t y[8];
                tmem_ld8(at, y);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = __float_as_uint(__uint_as_float(y[i]) * moves[8 * c + i].y);
                tmem_st8(at, y);
              }
            }
          if (!first) tmem_st_wait();
        }
        // weights, in three terms: 16 bytes a key and term for 16 rows, or for 8 the first two together
        if (j >= 2) wait(B_PV_DONE + (j & 1u), (j - 2) >> 1, 8);
        const uint32_t to = p_at + (j & 1u) * S::kWeights + static_cast<uint32_t>(group) * (3u * kKeys * 16u) + static_cast<uint32_t>(me) * 16u;
        if (chunks > 0) {
          uint32_t term[3][4] = {};
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (c < chunks) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {  // four rows
                uint32_t one[2], two[2];
                uint16_t three[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const int r = 8 * c + 4 * i + 2 * h;
                  const float w0 = ex2_approx(d[r]), w1 = ex2_approx(d[r + 1]);
                  l[r] = fmaf(w0, unbias, l[r]);
                  l[r + 1] = fmaf(w1, unbias, l[r + 1]);
                  three_terms(w0, w1, one[h], two[h], three[h]);
                }
                term[0][2 * c + i] = upper_bytes(one[0], one[1]);
                term[1][2 * c + i] = upper_bytes(two[0], two[1]);
                term[2][2 * c + i] = static_cast<uint32_t>(three[0]) | static_cast<uint32_t>(three[1]) << 16;
              }
            }
          if (kChunks == 1) {
            st_shared_v4(to, term[0][0], term[0][1], term[1][0], term[1][1]);
            st_shared_v4(to + kKeys * 16u, term[2][0], term[2][1], 0u, 0u);
          } else {
#pragma unroll
            for (int k = 0; k < 3; ++k) st_shared_v4(to + k * (kKeys * 16u), term[k][0], term[k][1], term[k][2], term[k][3]);
          }
        }
        if (__builtin_expect(tail && group == 0, 0)) {
          // values past the sequence's keys count as zero, NaN included
          const uint32_t slot_v = (2 * j + 1) % kSlots, v_at = ring + slot_v * kTile;
          wait(B_FULL + slot_v, (2 * j + 1) / kSlots, 9);
          const int len = pieces[item & 1u].len;
          for (int r = max(len - key0, 0) + (x >> 3); r < kKeys; r += 16)
            st_shared_v4(v_at + static_cast<uint32_t>(r * 128 + (x & 7) * 16), 0u, 0u, 0u, 0u);
        }
        if (__builtin_expect(tail && least < pieces[item & 1u].len, 0)) {
          // so does NaN among keys that some rows do not see, and the rows that do get it at the item's end.  (Each group looks before one
          // clears them.)
          const uint32_t slot_v = (2 * j + 1) % kSlots, v_at = ring + slot_v * kTile;
          wait(B_FULL + slot_v, (2 * j + 1) / kSlots, 9);
          const int r0 = max(least - key0, 0), r1 = min(pieces[item & 1u].len - key0, kKeys);
          auto place = [&](int r) { return v_at + static_cast<uint32_t>(r * 128 + (((me >> 4) ^ (r & 7)) << 4) + (me & 15)); };
          auto is_nan = [&](int r) {
            uint32_t code;
            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(code) : "r"(place(r)) : "memory");
            return (code & 0x7Fu) == 0x7Fu;
          };
          for (int r = r0; r < r1; ++r)
            if (is_nan(r)) nan_key = min(nan_key, key0 + r);
          groups_sync();
          if (group == 0)
            for (int r = r0; r < r1; ++r)
              if (is_nan(r)) asm volatile("st.shared.u8 [%0], %1;" ::"r"(place(r)), "r"(0u) : "memory");
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_P_FULL + (j & 1u)));
      }

      // ---- what the piece's keys came to
      {
        const float sum = row_sums<kRows>(l, lane);
        if ((lane & (32 / kRows - 1)) == 0) sums[(warp & 3) * kRows + lane / (32 / kRows)] = sum;
      }
      group_sync(group);
      const Piece p = pieces[item & 1u];
      const bool all = p.t0 == 0 && p.t1 == p.tiles, out = all && a.shared == 0;
      if (x < count) {
        const float den = (sums[x] + sums[kRows + x]) + (sums[2 * kRows + x] + sums[3 * kRows + x]);
        const Row row = rows[x];
        const float m = row.begun ? row.base : -INFINITY;
        const int in = group * kRows + x, r = p.block * R + in, token = r / a.group;
        const int64_t row_at = first_token(a, p.s) + token, place = row_at * a.hq + (p.head + lane_head) * a.group + r - token * a.group;
        OutRow to;
        to.limit = row.limit;
        to.factor = 1.0f;
        if (out) {
          const bool some = den > 0.0f || den != den;
          to.factor = some ? 1.0f / den : 0.0f;
          to.at = row_at * a.ld_o + (static_cast<int64_t>(p.head + lane_head) * a.group + r - token * a.group) * 128;
          if (a.lse && ok) a.lse[place] = some ? (m + log2f(den)) * 0.69314718055994531f : -INFINITY;
        } else {
          const int64_t slot = (2 * range + (p.at > lo ? 1 : 0)) * a.abreast + lane_head;  // (the item begins within the range)
          to.at = all ? (place + (is_shared(a, p.s) ? a.whole_rows : 0)) * kPart : (slot * R + in) * kPart;
          if (ok) *reinterpret_cast<float2*>((all ? w.whole : w.slots) + to.at + 128) = make_float2(m, den);
        }
        *reinterpret_cast<OutRow*>(rows + x) = to;
      }
      wait(B_PV_DONE + ((j - 1) & 1u), (j - 1) >> 1, 10);
      tc_fence_after();
      group_sync(group);
      float* parts = all ? w.whole : w.slots;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        uint32_t y[3][8];
#pragma unroll
        for (int k = 0; k < 3; ++k) tmem_ld8(out_lanes + k * S::kTerms + 8u * c, y[k]);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (8 * c + i >= count || !ok) break;
          const OutRow to = *reinterpret_cast<const OutRow*>(rows + 8 * c + i);
          const float sum = fmaf(__uint_as_float(y[2][i]), kThird, fmaf(__uint_as_float(y[1][i]), kSecond, __uint_as_float(y[0][i])));
          const float o = to.limit > nan_key ? NAN : sum * to.factor;
          if (out)
            a.O[to.at + me] = static_cast<uint16_t>(pack_bf16x2(o, 0.0f));
          else
            parts[to.at + me] = o;
        }
      }
      // the item's rows and O are read
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_Q_EMPTY + (item & 1u)));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmem);
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

// Parts of row r of entry s for key head `head`, every `warps`-th of them; true if one covers all keys.
__device__ __forceinline__ bool join_parts(const CachedArgs& a, const CachedWork& w, int s, int head, int r, const float* whole, int lane,
                                           int warp, int warps, Joined& j) {
  int start;
  const CachedHeader h = *w.head;
  const int64_t base = w.base[s];
  const int tiles = tiles_of(sequence(a, s, start));
  if (tiles == 0) return false;
  const int rows = a.rows_of_block, block = r / rows, sub = head / a.abreast;
  const int64_t begin = base + static_cast<int64_t>(block * (a.hkv / a.abreast) + sub) * units_of(tiles), tile0 = begin + kItem;
  // (within the workspace also where lengths have changed since the other kernel read them)
  const int64_t most = h.ranges - 1, first = min(range_of(tile0, h), most), last = min(range_of(tile0 + tiles - 1, h), most);
  if (first == last) {
    if (a.shared && warp == 0) j.add(whole, lane);
    return true;
  }
  const int64_t slot = static_cast<int64_t>(rows) * kPart;
  const float* row = w.slots + (head - sub * a.abreast) * slot + static_cast<int64_t>(r - block * rows) * kPart;
  if (warp == 0) j.add(row + (2 * first + (begin > range_begin(first, h) ? 1 : 0)) * a.abreast * slot, lane);
#pragma unroll 4
  for (int64_t i = first + 1 + warp; i <= last; i += warps) j.add(row + 2 * i * a.abreast * slot, lane);  // (these begin within the item)
  return false;
}

// A block for each row, of `warps` warps that share its parts.
__global__ void __launch_bounds__(32 * kJoinWarps) cached_join_kernel(const CachedArgs a, const CachedWork w) {
  __shared__ __align__(16) float parts[kJoinWarps][kPart];
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t i = blockIdx.x;
  const int64_t token = i / a.hq;
  const int qh = static_cast<int>(i - token * a.hq), head = qh / a.group, in_group = qh - head * a.group;
  const int s = static_cast<int>(token / a.t), t = static_cast<int>(token - static_cast<int64_t>(s) * a.t);
  Joined j;
  if (a.shared)
    join_parts(a, w, 0, head, static_cast<int>(token) * a.group + in_group, w.whole + (a.whole_rows + i) * kPart, lane, warp, warps, j);
  if (join_parts(a, w, s + a.shared, head, t * a.group + in_group, w.whole + i * kPart, lane, warp, warps, j) && !a.shared) return;
  if (warps > 1) {
    *reinterpret_cast<float4*>(&parts[warp][4 * lane]) = j.o;
    if (lane == 0) *reinterpret_cast<float2*>(&parts[warp][128]) = make_float2(j.m, j.l);
    __syncthreads();
    if (warp != 0) return;
    for (int x = 1; x < warps; ++x) j.add(parts[x], lane);
  }
  const bool some = j.l > 0.0f || j.l != j.l;
  const float inv = some ? 1.0f / j.l : 0.0f;
  *reinterpret_cast<uint2*>(a.O + token * a.ld_o + static_cast<int64_t>(qh) * 128 + 4 * lane) =
      make_uint2(pack_bf16x2(j.o.x * inv, j.o.y * inv), pack_bf16x2(j.o.z * inv, j.o.w * inv));
  if (lane == 0 && a.lse) a.lse[i] = some ? (j.m + log2f(j.l)) * 0.69314718055994531f : -INFINITY;
}

// ---- workspace

__host__ int64_t up256(int64_t n) { return (n + 255) / 256 * 256; }

struct Region {
  int64_t base, slots, whole, total;
};
Region region(const CachedArgs& a) {
  Region r;
  r.base = up256(static_cast<int64_t>(sizeof(CachedHeader)));
  r.slots = up256(r.base + (a.n + a.shared) * int64_t(8));
  r.whole = up256(r.slots + int64_t(2) * kSms * kBlocks * a.rows_of_block * kPart * 4);
  r.total = up256(r.whole + (a.shared ? 2 * a.whole_rows : 0) * kPart * 4);
  return r;
}
CachedWork work_at(void* ws, const CachedArgs& a) {
  const Region r = region(a);
  uint8_t* p = static_cast<uint8_t*>(ws);
  CachedWork w;
  w.head = reinterpret_cast<CachedHeader*>(p);
  w.base = reinterpret_cast<int64_t*>(p + r.base);
  w.slots = reinterpret_cast<float*>(p + r.slots);
  w.whole = reinterpret_cast<float*>(p + r.whole);
  return w;
}

template <int R>
cudaError_t launch_rows(const CUtensorMap& k, const CUtensorMap& v, const CachedArgs& a, const CachedWork& w, int sms, cudaStream_t st) {
  static std::atomic<bool> ready_of[kMaxDevices];  // the shared-memory opt-in, per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!ready_of[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(cached_attention_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<R>::kSmem);
    if (e != cudaSuccess) return e;
    ready_of[dev].store(true, std::memory_order_release);
  }
  const int blocks = (sms < kSms ? sms : kSms) * kBlocks;
  const dim3 grid(static_cast<unsigned>(blocks < a.abreast ? a.abreast : blocks));  // (a range of blocks at least)
  return launch_pdl(cached_attention_kernel<R>, grid, dim3(Shape<R>::kThreads), Shape<R>::kSmem, 1, st, k, v, a, w);
}

}  // namespace

void cached_shape(CachedArgs* a) {
  a->rows = a->t * a->group;
  a->whole_rows = int64_t(a->n) * a->t * a->hq;
  a->shared_rows = a->shared ? a->n * a->rows : 0;
  const int most = a->shared ? a->shared_rows : a->rows;
  a->rows_of_block = 8;
  while (a->rows_of_block < 32 && a->rows_of_block < most) a->rows_of_block *= 2;
  auto blocks = [&](int rows) { return static_cast<int32_t>((int64_t(rows) + a->rows_of_block - 1) / a->rows_of_block); };
  a->blocks = blocks(a->rows);
  a->shared_blocks = blocks(a->shared_rows);
  a->abreast = kMaxAbreast;
  while (a->hkv % a->abreast != 0) --a->abreast;
}

int64_t cached_scratch_bytes(const CachedArgs& a) { return region(a).total; }

cudaError_t launch_cached_attention(const CUtensorMap& k, const CUtensorMap& v, const CachedArgs& a, void* ws, int sms, cudaStream_t st) {
  const CachedWork w = work_at(ws, a);
  switch (a.rows_of_block) {
    case 8: return launch_rows<8>(k, v, a, w, sms, st);
    case 16: return launch_rows<16>(k, v, a, w, sms, st);
    default: return launch_rows<32>(k, v, a, w, sms, st);
  }
}

cudaError_t launch_cached_join(const CachedArgs& a, void* ws, cudaStream_t st) {
  // warps for a row: with few items each is cut into many parts
  const int64_t items = int64_t(a.hkv) * (int64_t(a.n) * a.blocks + a.shared_blocks);
  int warps = 1;
  while (warps < kJoinWarps && items * warps * 4 < kSms * kBlocks) warps *= 2;
  return launch_pdl(cached_join_kernel, dim3(static_cast<unsigned>(a.whole_rows)), dim3(static_cast<unsigned>(32 * warps)), 0, 1, st, a,
                    work_at(ws, a));
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
