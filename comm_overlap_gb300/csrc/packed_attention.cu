// packed_attention.cu -- causal attention of packed sequences with grouped query heads: prompts, chunks
// of prompts over a cache and single tokens over a cache in one call, head dimension 128.
//
// Sequence s has queries cu_q[s] .. cu_q[s + 1] - 1 (rows of Q) and k_len[s] keys from row k_start[s] of
// K and V; its queries are the last of its keys' positions.  A tile is 128 rows of the score matrix: TQ =
// 128 / G consecutive tokens times the G query heads that share a key/value head, row = token x G +
// head, so that a key block is read once for all G heads, and one decoded token fills G rows.
//
// Three kernels:
//  plan     (one block) checks the lengths, lists the work and sorts it, longest first.  An item is two
//           tiles (2 TQ tokens) of a sequence for one key/value head, over its key blocks of 128.  Items
//           longer than twice an even share of the whole work are cut along the keys into parts.
//  attend   (persistent, one CTA an SM) walks the list in a fixed back-and-forth order: O = softmax(scale Q
//           K^T + mask) V with an online softmax over the key blocks, as in attention.cu: scores and O in
//           TMEM, P in bf16 in the scores' columns, one MMA issuer per tile taking turns.
//  combine  adds the parts of cut items: each part left its unnormalised O, maximum and sum.
// Only keys of the sequence count: scores of rows past its end are masked by position and its last value
// tile is cleared past its end in shared memory, so whatever lies there (NaN included) has no effect.
//
// Bound: the exponentials of the softmax and its hand-offs for prompts; memory (K and V once per G heads) for
// single tokens.
#include <cuda_bf16.h>

#include <atomic>

#include "actfn.cuh"
#include "f32x2.cuh"
#include "ops.h"
#include "ptx.cuh"

namespace dm {

namespace {

__device__ int g_packed_err;

constexpr int kD = 128;                       // head dimension
constexpr int kBlk = 128;                     // rows of a tile, keys of a block
constexpr uint32_t kTile = kBlk * kD * 2;     // 32 KiB: one Q, K or V tile
constexpr uint32_t kHalf = kTile / 2;         // one 64-column (128-byte) swizzle panel
constexpr uint32_t kOBox = 32 * 64 * 2;       // 4 KiB: one warp's 32 rows x 64 columns of O
constexpr int kThreads = 384;                 // warps: 0 producer, 1 and 2 issuers, 3 idle, 4-7 and 8-11 softmax
// Registers a thread after the split: launched with 168, the first warpgroup gives up 104 and the softmax
// warpgroups take 48 each (64 x 128 + 216 x 256 <= 168 x 384): a row's 128 scores and 64 packed p stay in
// registers (16384-token prompt: 2420 us with 168 for all and a softmax that spills, 1510 us so).
constexpr int kRegsRoles = 64, kRegsSoftmax = 216;
static_assert(kRegsRoles * 128 + kRegsSoftmax * 256 <= 168 * kThreads, "more registers than the block was launched with");
constexpr int kSmem = 1024 + 1024 + 6 * static_cast<int>(kTile) + 8 * static_cast<int>(kOBox);
static_assert(kSmem <= 232448, "shared memory beyond the per-CTA limit");
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kDrainNs = 200000000ull;
constexpr int kPlanThreads = 1024;  // as many as the sort has bins

// per tile: Q, O free, drain, turn; per ring slot: K, V; per tile and ring slot (2 x + slot): their releases; per tile and
// score buffer (2 x + buffer, which half blocks use in turn): S, P, P V done.  (Two P V may be outstanding when a
// softmax warp waits for the later one: with one barrier for both, its parity could not tell them apart.)
enum : int {
  B_Q_FULL = 0, B_Q_EMPTY = 2, B_K_FULL = 4, B_K_EMPTY = 6, B_V_FULL = 10, B_V_EMPTY = 12, B_S_FULL = 16,
  B_P_FULL = 20, B_PV_DONE = 24, B_O_FREE = 28, B_DRAIN = 30, B_TURN = 32, B_COUNT = 34
};

// ---- work list, in the workspace
struct PackedHeader {
  int entries, splits, pad[62];
};
// One pair of tiles (or a part of it) for every key/value head.
struct __align__(16) PackedEntry {
  int q_row, qn;      // first query row; queries of the sequence from there on
  int k_row, klen;    // first key row, keys
  int pos0, b0, b1;   // key position of query q_row; key blocks b0 .. b1 - 1
  int slot;           // -1, or the first partial slot: head h, tile x use slot + 2 h + x
};
// A pair of tiles that was cut: parts of `len` blocks, part p in slots slot + p 2 Hkv + 2 h + x.
struct __align__(16) PackedSplit {
  int q_row, qn, pos0, len, slot, pad[3];
};

__host__ __device__ inline int64_t up(int64_t n, int64_t a) { return (n + a - 1) / a * a; }

struct PackedLayout {
  int64_t prefix, entries, splits, o, ml, total;
  int cap_entries, cap_splits, cap_slots;
};
// Bounds: the pairs of tiles of all sequences are at most Tq / (2 TQ) + n.  With an even share of
// total / (2 kSms) blocks (total over all heads), fewer than 2 kSms / Hkv pairs are longer than a share, and
// their parts over all heads are at most 4 kSms (a pair of e > share blocks has at most 2 e / share).
constexpr int kSms = 152;
__host__ inline PackedLayout packed_layout(int64_t tq, int64_t n, int tokens, int hkv, int64_t tk) {
  PackedLayout l;
  const int64_t pairs = tq / (2 * tokens) + n;
  const bool cut = (tk + kBlk - 1) / kBlk > kPackedMinPart;
  l.cap_splits = cut ? static_cast<int>(pairs < 2 * kSms / hkv + 1 ? pairs : 2 * kSms / hkv + 1) : 0;
  l.cap_slots = cut ? 8 * kSms : 0;
  l.cap_entries = static_cast<int>(pairs + (cut ? 4 * kSms / hkv + 1 : 0));
  l.prefix = sizeof(PackedHeader);
  l.entries = up(l.prefix + (n > kPlanThreads ? n * 4 : 0), 256);
  l.splits = up(l.entries + int64_t(l.cap_entries) * sizeof(PackedEntry), 256);
  l.o = up(l.splits + int64_t(l.cap_splits) * sizeof(PackedSplit), 1024);
  l.ml = l.o + int64_t(l.cap_slots) * kBlk * kD * 4;
  l.total = l.ml + int64_t(l.cap_slots) * 2 * kBlk * 4;
  return l;
}

struct PackedWork {
  PackedHeader* head;
  int* prefix;
  PackedEntry* entries;
  PackedSplit* splits;
  float* o;    // slot: [column / 4][row][4]
  float* ml;   // slot: maximum (log2 domain) of the 128 rows, then their sums
  int cap_entries, cap_splits, cap_slots;
};

// ---- plan -----------------------------------------------------------------------------------------

// Lengths of sequence s; a sequence whose rows leave the tensors gets none and is recorded.
__device__ __forceinline__ void seq_lengths(const PackedArgs& a, int s, int& q0, int& qlen, int& k0, int& klen) {
  q0 = a.cu_q[s];
  const int q1 = a.cu_q[s + 1];
  k0 = a.k_start[s];
  klen = a.k_len[s];
  qlen = q1 - q0;
  if (q0 < 0 || q1 < q0 || q1 > a.tq || k0 < 0 || klen < 0 || klen > a.tk || k0 > a.tk - klen) {
    atomicCAS(&g_packed_err, 0, kPackedBadLengths);
    qlen = klen = k0 = q0 = 0;
  }
}

// Key blocks that the queries [tok0, tok1) of a sequence see.
__device__ __forceinline__ int seen_blocks(int qlen, int klen, int tok1) {
  const int last = klen - qlen + min(tok1, qlen) - 1;
  return last < 0 ? 0 : (last >> 7) + 1;
}

__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {  // exclusive
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the previous call's sums are read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  total = warp_sums[31];
  return x - v + (warp > 0 ? warp_sums[warp - 1] : 0);
}

// A pair of tiles: its sequence's lengths, its first token, the key blocks it sees.
struct PackedPair {
  int q0, qlen, k0, klen, tok0, e;
};

// The kernel is a chain of short dependent steps, so each thread keeps its first pair in registers, the totals are
// added by warp before they meet in shared memory, and the sequences' offsets are searched there when they
// fit (9 - 17 us before, with a pair's lengths looked up for each step and one atomic a pair).
__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(const PackedArgs a, const PackedWork w) {
  constexpr int kBins = 1024;
  __shared__ int warp_sums[32];
  __shared__ int bins[kBins];
  __shared__ int near_prefix[kPlanThreads];
  __shared__ unsigned long long s_total;
  __shared__ int s_max, s_slots, s_splits, s_bad;
  const int tid = threadIdx.x, span = 2 * a.tokens;
  if (tid == 0) {
    s_total = 0;
    s_max = s_slots = s_splits = s_bad = 0;
  }
  for (int i = tid; i < kBins; i += kPlanThreads) bins[i] = 0;
  pdl_launch();
  pdl_wait();
  // pairs of tiles before each sequence
  const bool near = a.n <= kPlanThreads;
  int pairs = 0;
  for (int base = 0; base < a.n; base += kPlanThreads) {
    const int s = base + tid;
    int q0, qlen = 0, k0, klen;
    if (s < a.n) seq_lengths(a, s, q0, qlen, k0, klen);
    int total;
    const int before = pairs + block_scan((qlen + span - 1) / span, warp_sums, total);
    if (s < a.n) (near ? near_prefix : w.prefix)[s] = before;
    pairs += total;
  }
  __syncthreads();
  const int* prefix = near ? near_prefix : w.prefix;
  // pair i belongs to the last sequence that begins at or before it
  auto pair_of = [&](int i) {
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= i) lo = mid; else hi = mid - 1;
    }
    PackedPair p;
    seq_lengths(a, lo, p.q0, p.qlen, p.k0, p.klen);
    p.tok0 = (i - prefix[lo]) * span;
    p.e = seen_blocks(p.qlen, p.klen, p.tok0 + span);
    return p;
  };
  PackedPair first = {};
  if (tid < pairs) first = pair_of(tid);
  unsigned long long mine = static_cast<unsigned long long>(first.e);
  int most = first.e;
  for (int i = tid + kPlanThreads; i < pairs; i += kPlanThreads) {
    const int e = pair_of(i).e;
    mine += static_cast<unsigned long long>(e);
    most = max(most, e);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mine += __shfl_xor_sync(0xFFFFFFFFu, mine, o);
    most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
  }
  if ((tid & 31) == 0 && most > 0) {
    atomicAdd(&s_total, mine);
    atomicMax(&s_max, most);
  }
  __syncthreads();
  // even share of the blocks, twice per SM; parts of at least kPackedMinPart blocks
  const unsigned long long total = s_total * static_cast<unsigned long long>(a.hkv);
  const unsigned long long even = (total + 2 * kSms - 1) / (2 * kSms);
  int share = even > 0x7FFFFFFFull ? 0x7FFFFFFF : static_cast<int>(even);
  if (share < kPackedMinPart) share = kPackedMinPart;
  if (w.cap_slots == 0) share = 0x7FFFFFFF;
  auto parts_of = [&](int e, int& len) {
    len = e;
    if (e <= share) return 1;
    const int parts = (e + share - 1) / share;
    len = (e + parts - 1) / parts;
    return (e + len - 1) / len;
  };
  int shift = 0;
  while ((min(s_max, share) >> shift) >= kBins) ++shift;
  // longest first: counting sort by blocks (order within a bin is of no consequence)
  for (int i = tid; i < pairs; i += kPlanThreads) {
    const int e = i == tid ? first.e : pair_of(i).e;
    int len;
    const int parts = parts_of(e, len);
    if (parts > 1) atomicAdd(&bins[kBins - 1 - (len >> shift)], parts - 1);
    atomicAdd(&bins[kBins - 1 - ((e - (parts - 1) * len) >> shift)], 1);
  }
  __syncthreads();
  int count;
  const int start = block_scan(bins[tid], warp_sums, count);
  bins[tid] = start;
  __syncthreads();
  for (int i = tid; i < pairs; i += kPlanThreads) {
    const PackedPair p = i == tid ? first : pair_of(i);
    int len;
    const int parts = parts_of(p.e, len);
    PackedEntry en;
    en.q_row = p.q0 + p.tok0;
    en.qn = p.qlen - p.tok0;
    en.k_row = p.k0;
    en.klen = p.klen;
    en.pos0 = p.klen - p.qlen + p.tok0;
    int slot = -1;
    if (parts > 1) {
      slot = atomicAdd(&s_slots, parts * 2 * a.hkv);
      const int sp = atomicAdd(&s_splits, 1);
      if (sp < w.cap_splits && slot + parts * 2 * a.hkv <= w.cap_slots) {
        PackedSplit ps;
        ps.q_row = en.q_row;
        ps.qn = en.qn;
        ps.pos0 = en.pos0;
        ps.len = len;
        ps.slot = slot;
        w.splits[sp] = ps;
      } else {
        s_bad = 1;
        continue;
      }
    }
    for (int k = 0; k < parts; ++k) {
      en.b0 = k * len;
      en.b1 = min(p.e, en.b0 + len);
      en.slot = parts > 1 ? slot + k * 2 * a.hkv : -1;
      const int at = atomicAdd(&bins[kBins - 1 - ((en.b1 - en.b0) >> shift)], 1);
      if (at < w.cap_entries)
        w.entries[at] = en;
      else
        s_bad = 1;
    }
  }
  __syncthreads();
  if (tid == 0) {
    // beyond the bounds of the workspace only with overlapping sequences, which are refused
    if (s_bad) atomicCAS(&g_packed_err, 0, kPackedBadLengths);
    w.head->entries = s_bad ? 0 : count;
    w.head->splits = s_bad ? 0 : s_splits;
  }
}

// ---- attend ---------------------------------------------------------------------------------------

// the largest of three (a NaN score makes its own p NaN and need not show in the maximum)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// As mbar_wait (bounded), but polling: the thread is never suspended.
__device__ __forceinline__ bool mbar_poll(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err, int site) {
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((it & 1023u) == 1023u) {
      if (*abort_flag) return false;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > kWaitTimeoutNs) {
        *abort_flag = 1;
        atomicCAS(err, 0, site);
        return false;
      }
    }
  }
}

struct Item {
  int hk, q_row, qn, k_row, klen, pos0, b0, slot;
  int e0, e1;   // tile x attends to half blocks (64 keys) 2 b0 .. e_x - 1 (none: e_x <= 2 b0)
  int last;     // blocks b0 .. last - 1 are loaded
  __device__ int e(int x) const { return x ? e1 : e0; }
  __device__ bool active(int x) const { return e(x) > 2 * b0; }
  __device__ bool both() const { return e0 > 2 * b0 && e1 > 2 * b0; }
};

// The k-th item of this CTA: the list in rounds of gridDim.x, every other round backwards.
__device__ __forceinline__ bool item_at(const PackedArgs& a, const PackedWork& w, int total, int k, Item& it) {
  const int g = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
  const int64_t i = static_cast<int64_t>(k) * g + ((k & 1) ? g - 1 - c : c);
  if (i >= total) return false;
  const int en = static_cast<int>(i) / a.hkv;
  it.hk = static_cast<int>(i) - en * a.hkv;
  const int4* p = reinterpret_cast<const int4*>(w.entries + en);
  const int4 u = p[0], v = p[1];
  it.q_row = u.x;
  it.qn = u.y;
  it.k_row = u.z;
  it.klen = u.w;
  it.pos0 = v.x;
  it.b0 = v.y;
  it.slot = v.w < 0 ? -1 : v.w + 2 * it.hk;
  // the last position that each tile's queries see
  const int l0 = it.pos0 + min(a.tokens, it.qn) - 1, l1 = it.pos0 + min(2 * a.tokens, it.qn) - 1;
  it.e0 = min(2 * v.z, l0 < 0 ? 0 : (l0 >> 6) + 1);
  it.e1 = it.qn > a.tokens ? min(2 * v.z, l1 < 0 ? 0 : (l1 >> 6) + 1) : 0;
  it.last = (max(it.e0, it.e1) + 1) >> 1;
  if (it.last < it.b0) it.last = it.b0;
  return true;
}

__global__ void __launch_bounds__(kThreads, 1)
    packed_attention_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV, const PackedArgs a, const PackedWork w) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + 512);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + 516);
  const uint32_t bar0 = smem_u32(smem);
  auto bar = [bar0](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  const uint32_t sQ = smem_u32(smem + 1024), sK = sQ + 2 * kTile, sV = sQ + 4 * kTile, sO = sQ + 6 * kTile;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* err = &g_packed_err;

  if (threadIdx.x == 0) {
    for (int i = 0; i < B_COUNT; ++i)
      mbar_init(bar(i), ((i >= B_P_FULL && i < B_PV_DONE) || i == B_O_FREE || i == B_O_FREE + 1) ? 4 : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  pdl_launch();
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int total = w.head->entries * a.hkv;

  if (warp < 4)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRoles));
  else
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer
      uint32_t gb = 0;      // ring position of the item's first key block
      uint32_t nq[2] = {0, 0};
      // ring slot b's block: bit 2 b + x set if tile x consumes it (cons); parity of the blocks of slot b
      // that tile x consumed so far (upar)
      uint32_t cons = 0, upar = 0;
      const uint32_t q_bytes = static_cast<uint32_t>(a.tokens * a.group) * 128u;
      bool ok = true;
      Item it;
      for (int k = 0; ok && item_at(a, w, total, k, it); ++k) {
        for (int x = 0; x < 2 && ok; ++x) {
          if (!it.active(x)) continue;
          // tile x's Q buffer is free once its previous item's last Q K^T has completed
          if (nq[x] > 0)
            ok = mbar_wait(bar(B_Q_EMPTY + x), (nq[x] - 1) & 1u, abort_flag, err, a.err_site + 1);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(B_Q_FULL + x), 2 * q_bytes);
          const int row = it.q_row + x * a.tokens;
          tma_load_4d(sQ + x * kTile, &tmQ, bar(B_Q_FULL + x), 0, 0, it.hk, row);
          tma_load_4d(sQ + x * kTile + kHalf, &tmQ, bar(B_Q_FULL + x), 64, 0, it.hk, row);
          ++nq[x];
        }
        for (int j = it.b0; ok && j < it.last; ++j) {
          const uint32_t r = gb + static_cast<uint32_t>(j - it.b0);
          const int b = static_cast<int>(r & 1u);
          const int row = it.k_row + j * kBlk;
          // the slot is refilled once every tile that consumed its previous block has released it
          for (int x = 0; x < 2 && ok; ++x)
            if ((cons >> (2 * b + x)) & 1u)
              ok = mbar_wait(bar(B_K_EMPTY + 2 * x + b), ((upar >> (2 * b + x)) & 1u) ^ 1u, abort_flag, err,
                             a.err_site + 2);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(B_K_FULL + b), kTile);
          tma_load_3d(sK + b * kTile, &tmK, bar(B_K_FULL + b), 0, it.hk, row);
          tma_load_3d(sK + b * kTile + kHalf, &tmK, bar(B_K_FULL + b), 64, it.hk, row);
          for (int x = 0; x < 2 && ok; ++x)
            if ((cons >> (2 * b + x)) & 1u)
              ok = mbar_wait(bar(B_V_EMPTY + 2 * x + b), ((upar >> (2 * b + x)) & 1u) ^ 1u, abort_flag, err,
                             a.err_site + 3);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(B_V_FULL + b), kTile);
          tma_load_3d(sV + b * kTile, &tmV, bar(B_V_FULL + b), 0, it.hk, row);
          tma_load_3d(sV + b * kTile + kHalf, &tmV, bar(B_V_FULL + b), 64, it.hk, row);
          const uint32_t users = (2 * j < it.e0 ? 1u : 0u) | (2 * j < it.e1 ? 2u : 0u);
          cons = (cons & ~(3u << (2 * b))) | (users << (2 * b));
          upar ^= users << (2 * b);
        }
        gb += static_cast<uint32_t>(it.last - it.b0);
      }
      if (!ok) {
        // let the copies still in flight land before the CTA leaves
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 100000ull) {
        }
      }
    }
    __syncwarp();
  } else if (warp < 3) {
    {
      // ---------------- MMA issuer of tile x (the warp walks the work, one elected lane issues).  Scores are made
      // in half blocks of 64 keys, two of them in flight (buffers of 64 TMEM columns, P in the first 32), so that
      // the softmax of one runs while the tensor core makes the next: S of half blocks 0 and 1 first, then for
      // each half block n P V of it and S of n + 2, in the same buffer.  In items where both tiles work the
      // issuers alternate, half block by half block; a tile that has no work left passes its turn on.  Elsewhere
      // the one with work needs no turn.
      const uint32_t x = static_cast<uint32_t>(warp) - 1u;
      constexpr uint32_t kIdQK = idesc_bf16_f32(kBlk, 64, false, false);
      constexpr uint32_t kIdPV = idesc_bf16_f32(kBlk, kD, false, true);
      const uint64_t dQ = sdesc_sw128(sQ + x * kTile, 16, 1024), dK0 = sdesc_sw128(sK, 16, 1024),
                     dV0 = sdesc_sw128(sV, kHalf, 1024);
      const uint32_t tS = tmem_base + 128u * x, tO = tmem_base + 256u + 128u * x;
      const bool one = elect_one();
      uint32_t gb = 0, nq = 0, np = 0, turns = 0;  // ring position; items and half blocks of this tile; turns received
      // S of half block h (of ring position gb) into the buffer of half block count n
      auto qk = [&](int h, uint32_t n) {
        const uint64_t dk = dK0 + ((static_cast<uint64_t>((gb + (static_cast<uint32_t>(h) >> 1)) & 1u) * kTile + (h & 1) * 8192u) >> 4);
#pragma unroll
        for (int kk = 0; kk < kD / 16; ++kk) {
          const uint64_t off = (static_cast<uint64_t>(kk >> 2) * kHalf + static_cast<uint64_t>(kk & 3) * 32u) >> 4;
          umma_bf16(tS + 64u * (n & 1u), dQ + off, dk + off, kIdQK, static_cast<uint32_t>(kk != 0));
        }
      };
      auto pv = [&](int h, uint32_t n, bool first) {
        const uint64_t dv = dV0 + ((static_cast<uint64_t>((gb + (static_cast<uint32_t>(h) >> 1)) & 1u) * kTile + (h & 1) * 8192u) >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16_tmem_a(tO, tS + 64u * (n & 1u) + 8u * kk, dv + ((static_cast<uint64_t>(kk) * 2048u) >> 4), kIdPV,
                           static_cast<uint32_t>(!first || kk != 0));
      };
      bool ok = true, shared_before = false;
      auto take_turn = [&](bool needed) -> bool {
        if (!needed) return true;
        if (!mbar_wait(bar(B_TURN + x), turns & 1u, abort_flag, err, a.err_site + 4)) return false;
        ++turns;
        return true;
      };
      auto k_ready = [&](int h) {
        const uint32_t r = gb + (static_cast<uint32_t>(h) >> 1);
        return mbar_wait(bar(B_K_FULL + (r & 1u)), (r >> 1) & 1u, abort_flag, err, a.err_site + 6);
      };
      Item it;
      for (int k = 0; ok && item_at(a, w, total, k, it); ++k) {
        const bool two = it.both();
        const int n = it.e(static_cast<int>(x)) - 2 * it.b0, most = max(it.e0, it.e1) - 2 * it.b0;  // half blocks: this tile's, all
        const uint32_t blocks = static_cast<uint32_t>(it.last - it.b0);
        if (n > 0) {
          // after S of half block h: its block is released once its last half block of this tile is done
          auto made_s = [&](int h, uint32_t c) {
            umma_commit(bar(B_S_FULL + 2 * x + (c & 1u)));
            if ((h & 1) || h == n - 1) umma_commit(bar(B_K_EMPTY + 2 * x + ((gb + (static_cast<uint32_t>(h) >> 1)) & 1u)));
            if (h == n - 1) umma_commit(bar(B_Q_EMPTY + x));
          };
          // the first turn ever is tile 0's
          if (!mbar_wait(bar(B_Q_FULL + x), nq & 1u, abort_flag, err, a.err_site + 5) || !k_ready(0) ||
              !take_turn(two && (x == 1 || shared_before))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (one) {
            qk(0, np);
            made_s(0, np);
            if (n > 1) {
              qk(1, np + 1);
              made_s(1, np + 1);
            }
            if (two) mbar_arrive(bar(B_TURN + (x ^ 1u)));
          }
          for (int h = 0; ok && h < most; ++h) {
            if (h >= n) {  // the other tile alone
              ok = take_turn(two);
              if (ok && two && one) mbar_arrive(bar(B_TURN + (x ^ 1u)));
              continue;
            }
            const uint32_t r = gb + (static_cast<uint32_t>(h) >> 1);
            // the waits that are usually over first, the softmax hand-off (the critical path) last
            if (!mbar_wait(bar(B_V_FULL + (r & 1u)), (r >> 1) & 1u, abort_flag, err, a.err_site + 7) ||
                (h + 2 < n && !k_ready(h + 2)) ||
                // the item's first P V overwrites O: the previous item's must be read
                (h == 0 && nq > 0 && !mbar_wait(bar(B_O_FREE + x), (nq - 1) & 1u, abort_flag, err, a.err_site + 8)) ||
                !take_turn(two) || !mbar_poll(bar(B_P_FULL + 2 * x + (np & 1u)), (np >> 1) & 1u, abort_flag, err, a.err_site + 9)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (one) {
              pv(h, np, h == 0);
              umma_commit(bar(B_PV_DONE + 2 * x + (np & 1u)));
              if ((h & 1) || h == n - 1) umma_commit(bar(B_V_EMPTY + 2 * x + (r & 1u)));
              if (h + 2 < n) {
                qk(h + 2, np);  // overwrites P only after the product above (issue order)
                made_s(h + 2, np);
              }
              if (two) mbar_arrive(bar(B_TURN + (x ^ 1u)));
            }
            ++np;
          }
          ++nq;
        }
        shared_before |= two;
        gb += blocks;
      }
      if (one) umma_commit(bar(B_DRAIN + x));
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(bar(B_DRAIN + x), 0) && global_timer_ns() - t0 <= kDrainNs) {
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------- softmax warps of tile x, one row a thread
    const int x = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t lq = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem_base + lq + 128u * x, tO = tmem_base + lq + 256u + 128u * x;
    const uint32_t obox = sO + static_cast<uint32_t>(warp - 4) * kOBox;
    const int rows = a.tokens * a.group;
    // row / group for rows below 128 (exact: the rounding of the factor adds less than 1 / group)
    const uint32_t inv_group = (65536u + static_cast<uint32_t>(a.group) - 1u) / static_cast<uint32_t>(a.group);
    auto token_of = [inv_group](int r) { return static_cast<int>((static_cast<uint32_t>(r) * inv_group) >> 16); };
    const int tok = token_of(row);
    uint32_t cb = 0, gb = 0;  // half blocks this tile has processed; ring position
    bool ok = true;
    Item it;
    for (int k = 0; ok && item_at(a, w, total, k, it); ++k) {
      const int e = it.e(x), first = 2 * it.b0, klen = it.klen;
      // the last key position that this row sees (none for rows outside)
      const int lim = row < rows && tok < it.qn - x * a.tokens ? min(it.pos0 + x * a.tokens + tok, klen - 1) : -1;
      float m_run = -INFINITY, l_run = 0.0f;
      for (int j = first; ok && j < e; ++j, ++cb) {
        const uint32_t tB = tS + 64u * (cb & 1u);
        ok = mbar_wait(bar(B_S_FULL + 2 * x + (cb & 1u)), (cb >> 1) & 1u, abort_flag, err, a.err_site + 10);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t sr[2][32];
        tmem_ld32(tB, sr[0]);
        tmem_ld32(tB + 32u, sr[1]);
        tmem_ld_wait();
        const int rel = lim - j * 64;  // columns above it are masked
        if (__any_sync(0xFFFFFFFFu, rel < 63)) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c > rel) sr[c >> 5][c & 31] = __float_as_uint(-INFINITY);
        }
        float m4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) m4[i] = -INFINITY;
#pragma unroll
        for (int c = 0; c < 64; c += 2)
          m4[(c >> 1) & 3] = max3(m4[(c >> 1) & 3], __uint_as_float(sr[c >> 5][c & 31]),
                                  __uint_as_float(sr[c >> 5][(c & 31) + 1]));
        const float top = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
        // running maximum in the log2 domain, raised when some row of the warp would pass it by more than
        // 8 (p <= 2^8 otherwise); O and the sum are then rescaled.  A row that has seen no key keeps
        // -inf, and zero stands in for it so that its p are 0 and not NaN.
        const float cand = fmaxf(m_run, top * a.scale_log2);
        const bool raise = __any_sync(0xFFFFFFFFu, cand > m_run + 8.0f) || j == first;
        const float mx = raise ? cand : m_run;
        const float base = mx == -INFINITY ? 0.0f : mx;
        const float alpha = raise ? ex2_approx(m_run - base) : 1.0f;
        uint64_t l4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) l4[i] = f2(0.0f, 0.0f);
        const uint64_t sc2 = f2(a.scale_log2, a.scale_log2), nmx2 = f2(-base, -base);
        uint32_t pk[32];
        // p = 2^(score - maximum), two columns at a time
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const int i = 2 * c;
          float p0, p1;
          f2_split(fma_f2(f2(__uint_as_float(sr[i >> 5][i & 31]), __uint_as_float(sr[i >> 5][(i & 31) + 1])), sc2, nmx2), p0, p1);
          p0 = ex2_approx(p0);
          p1 = ex2_approx(p1);
          l4[c & 3] = add_f2(l4[c & 3], f2(p0, p1));
          pk[c] = pack_bf16x2(p0, p1);
        }
        tmem_st32(tB, pk);  // P -> the first 32 columns of its scores
        float l0, l1;
        f2_split(add_f2(add_f2(l4[0], l4[1]), add_f2(l4[2], l4[3])), l0, l1);
        l_run = l_run * alpha + (l0 + l1);
        m_run = mx;
        if (j > first && raise) {
          // O is free once the previous half block's P V has completed
          ok = mbar_wait(bar(B_PV_DONE + 2 * x + ((cb - 1u) & 1u)), ((cb - 1u) >> 1) & 1u, abort_flag, err, a.err_site + 13);
          if (!__all_sync(0xFFFFFFFFu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + static_cast<uint32_t>(c * 32), o);
            tmem_ld_wait();
            const uint64_t al2 = f2(alpha, alpha);
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              float v0, v1;
              f2_split(mul_f2(f2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), al2), v0, v1);
              o[i] = __float_as_uint(v0);
              o[i + 1] = __float_as_uint(v1);
            }
            tmem_st32(tO + static_cast<uint32_t>(c * 32), o);
          }
        }
        if ((j + 1) * 64 > klen) {
          // the half block's value rows past the sequence: cleared before the product reads them (0 x NaN)
          const uint32_t r = gb + (static_cast<uint32_t>(j - first) >> 1);
          ok = mbar_wait(bar(B_V_FULL + (r & 1u)), (r >> 1) & 1u, abort_flag, err, a.err_site + 11);
          if (!__all_sync(0xFFFFFFFFu, ok)) {
            ok = false;
            break;
          }
          const uint32_t v = sV + (r & 1u) * kTile + static_cast<uint32_t>(j & 1) * 8192u;
          for (int c = klen - j * 64 + (row >> 3); c < 64; c += 16)
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h)
              st_shared_v4(v + h * kHalf + static_cast<uint32_t>(c) * 128u + (static_cast<uint32_t>(row) & 7u) * 16u, 0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_P_FULL + 2 * x + (cb & 1u)));
      }
      if (!ok) break;
      item_at(a, w, total, k, it);  // again, rather than kept in registers through the blocks
      gb += static_cast<uint32_t>(it.last - it.b0);
      const int live = min(a.tokens, it.qn - x * a.tokens);  // tokens of the tile that exist
      const bool row_ok = row < rows && tok < live;
      if (e > first) {
        ok = mbar_wait(bar(B_PV_DONE + 2 * x + ((cb - 1u) & 1u)), ((cb - 1u) >> 1) & 1u, abort_flag, err, a.err_site + 12);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
      } else if (it.slot >= 0 || live <= 0) {
        continue;  // nothing of this tile in this part
      }
      const bool any = live * a.group > quarter * 32;  // some row of the warp exists
      if (it.slot >= 0) {
        // a part: unnormalised O, maximum and sum
        float* so = w.o + static_cast<int64_t>(it.slot + x) * (kBlk * kD);
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          if (any) {
            tmem_ld32(tO + static_cast<uint32_t>(c * 32), o);
            tmem_ld_wait();
          }
          if (c == 3) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_O_FREE + x));
          }
          if (row_ok) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(so + ((c * 8 + i) * kBlk + row) * 4) =
                  make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        if (row_ok) {
          float* ml = w.ml + static_cast<int64_t>(it.slot + x) * (2 * kBlk);
          ml[row] = m_run;
          ml[kBlk + row] = l_run;
        }
        continue;
      }
      // O / sum -> bf16, 64 columns at a time through this warp's box (32 rows x 128 bytes, 16-byte piece
      // j of row r at j ^ (r % 8)), then row by row with eight lanes each; rows without keys are zero
      const float inv = l_run > 0.0f || l_run != l_run ? 1.0f / l_run : 0.0f;
      if (row_ok && a.lse)
        a.lse[static_cast<int64_t>(it.q_row + x * a.tokens + tok) * a.hq + it.hk * a.group + (row - tok * a.group)] =
            l_run > 0.0f || l_run != l_run ? (m_run + log2f(l_run)) * 0.69314718055994531f : -INFINITY;
#pragma unroll 1
      for (int h2 = 0; h2 < 2; ++h2) {
        uint32_t o[2][32];
        if (e > first && any) {
          tmem_ld32(tO + static_cast<uint32_t>(h2 * 64), o[0]);
          tmem_ld32(tO + static_cast<uint32_t>(h2 * 64 + 32), o[1]);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[0][i] = o[1][i] = 0u;
        }
        if (h2 == 1 && e > first) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_O_FREE + x));
        }
        if (!any) continue;
        __syncwarp();  // the box's previous contents are read
        const uint32_t box = obox + static_cast<uint32_t>(lane) * 128u;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t unit = static_cast<uint32_t>(c * 4 + i);
            st_shared_v4(box + ((unit ^ (static_cast<uint32_t>(lane) & 7u)) << 4),
                         pack_bf16x2(__uint_as_float(o[c][8 * i]) * inv, __uint_as_float(o[c][8 * i + 1]) * inv),
                         pack_bf16x2(__uint_as_float(o[c][8 * i + 2]) * inv, __uint_as_float(o[c][8 * i + 3]) * inv),
                         pack_bf16x2(__uint_as_float(o[c][8 * i + 4]) * inv, __uint_as_float(o[c][8 * i + 5]) * inv),
                         pack_bf16x2(__uint_as_float(o[c][8 * i + 6]) * inv, __uint_as_float(o[c][8 * i + 7]) * inv));
          }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rb = i * 4 + (lane >> 3), rt = quarter * 32 + rb, t = token_of(rt);
          const uint4 v = ld_shared_v4(obox + static_cast<uint32_t>(rb) * 128u +
                                       (((static_cast<uint32_t>(lane) & 7u) ^ (static_cast<uint32_t>(rb) & 7u)) << 4));
          if (rt < rows && t < live) {
            uint16_t* dst = a.O + static_cast<int64_t>(it.q_row + x * a.tokens + t) * a.ld_o +
                            static_cast<int64_t>(it.hk * a.group + (rt - t * a.group)) * kD + h2 * 64 + (lane & 7) * 8;
            *reinterpret_cast<uint4*>(dst) = v;
          }
        }
      }
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

// ---- combine --------------------------------------------------------------------------------------
// Block (split, key/value head, tile): with m = max m_p and c_p = 2^(m_p - m) over the parts p in order,
// O = sum c_p O_p / sum c_p l_p, lse = ln 2 (m + log2(sum c_p l_p)).
__global__ void __launch_bounds__(256) packed_combine_kernel(const PackedArgs a, const PackedWork w) {
  pdl_launch();
  pdl_wait();
  if (static_cast<int>(blockIdx.x) >= w.head->splits) return;
  const PackedSplit s = w.splits[blockIdx.x];
  const int hk = blockIdx.y, x = blockIdx.z;
  const int live = min(a.tokens, s.qn - x * a.tokens);
  if (live <= 0) return;
  const int last = s.pos0 + x * a.tokens + live - 1, e = last < 0 ? 0 : (last >> 7) + 1;
  const int parts = (e + s.len - 1) / s.len, rows = live * a.group;
  const int64_t step = 2 * a.hkv, first = s.slot + 2 * hk + x;
  for (int i = threadIdx.x; i < rows * 32; i += 256) {
    const int row = i % rows, c = i / rows;  // piece c: columns 4 c .. 4 c + 3
    float m = -INFINITY;
    for (int p = 0; p < parts; ++p) m = fmaxf(m, w.ml[(first + p * step) * (2 * kBlk) + row]);
    float l = 0.0f, o0 = 0.0f, o1 = 0.0f, o2 = 0.0f, o3 = 0.0f;
    const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      const float* ml = w.ml + (first + p * step) * (2 * kBlk);
      const float f = exp2f(ml[row] - base);
      const float4 v = *reinterpret_cast<const float4*>(w.o + (first + p * step) * (kBlk * kD) + (c * kBlk + row) * 4);
      l = fmaf(f, ml[kBlk + row], l);
      o0 = fmaf(f, v.x, o0);
      o1 = fmaf(f, v.y, o1);
      o2 = fmaf(f, v.z, o2);
      o3 = fmaf(f, v.w, o3);
    }
    const bool some = l > 0.0f || l != l;
    const float inv = some ? 1.0f / l : 0.0f;
    const int t = row / a.group;
    const int64_t token = s.q_row + x * a.tokens + t;
    const int head = hk * a.group + row - t * a.group;
    *reinterpret_cast<uint2*>(a.O + token * a.ld_o + static_cast<int64_t>(head) * kD + c * 4) =
        make_uint2(pack_bf16x2(o0 * inv, o1 * inv), pack_bf16x2(o2 * inv, o3 * inv));
    if (c == 0 && a.lse) a.lse[token * a.hq + head] = some ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
  }
}

PackedWork packed_work(const PackedArgs& a, void* ws) {
  const PackedLayout l = packed_layout(a.tq, a.n, a.tokens, a.hkv, a.tk);
  uint8_t* p = static_cast<uint8_t*>(ws);
  PackedWork w;
  w.head = reinterpret_cast<PackedHeader*>(p);
  w.prefix = reinterpret_cast<int*>(p + l.prefix);
  w.entries = reinterpret_cast<PackedEntry*>(p + l.entries);
  w.splits = reinterpret_cast<PackedSplit*>(p + l.splits);
  w.o = reinterpret_cast<float*>(p + l.o);
  w.ml = reinterpret_cast<float*>(p + l.ml);
  w.cap_entries = l.cap_entries;
  w.cap_splits = l.cap_splits;
  w.cap_slots = l.cap_slots;
  return w;
}

}  // namespace

int64_t packed_scratch_bytes(int64_t tq, int64_t n, int hq, int hkv, int64_t tk) {
  return packed_layout(tq, n, kBlk / (hq / hkv), hkv, tk).total;
}

cudaError_t launch_packed_plan(const PackedArgs& a, void* ws, cudaStream_t st) {
  return launch_pdl(packed_plan_kernel, dim3(1), dim3(kPlanThreads), 0, 1, st, a, packed_work(a, ws));
}

cudaError_t launch_packed_attention(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                    const PackedArgs& a, void* ws, int sms, cudaStream_t st) {
  static std::atomic<bool> ready_of[kMaxDevices];  // the shared-memory opt-in, per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!ready_of[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(packed_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    ready_of[dev].store(true, std::memory_order_release);
  }
  const PackedWork w = packed_work(a, ws);
  const int64_t most = int64_t(w.cap_entries) * a.hkv;
  const int grid = static_cast<int>(most < sms ? most : sms);
  return launch_pdl(packed_attention_kernel, dim3(grid), dim3(kThreads), kSmem, 1, st, q, k, v, a, w);
}

bool packed_may_cut(const PackedArgs& a) {
  return packed_layout(a.tq, a.n, a.tokens, a.hkv, a.tk).cap_splits > 0;
}

cudaError_t launch_packed_combine(const PackedArgs& a, void* ws, cudaStream_t st) {
  const PackedWork w = packed_work(a, ws);
  return launch_pdl(packed_combine_kernel, dim3(static_cast<unsigned>(w.cap_splits), static_cast<unsigned>(a.hkv), 2), dim3(256), 0, 1,
                    st, a, w);
}

cudaError_t take_packed_error(int* code) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_packed_err, sizeof(int));
  if (e != cudaSuccess) return e;
  *code = v;
  if (v != 0) {
    const int zero = 0;
    e = cudaMemcpyToSymbol(g_packed_err, &zero, sizeof(int));
  }
  return e;
}

}  // namespace dm
