// packed_attention.cu -- causal attention of packed sequences with grouped query heads: prompts, chunks
// of prompts over a cache and single tokens over a cache in one call, head dimension 128.
//
// Sequence s has queries cu_q[s] .. cu_q[s + 1] - 1 (rows of Q) and k_len[s] keys from row k_start[s] of
// K and V; its queries are the last of its keys' positions.  A tile is 128 rows of the score matrix: TQ =
// 128 / G consecutive tokens times the G query heads that share a key/value head, row = token x G +
// head, so that a key block is read once for all G heads, and one decoded token fills G rows.
//
// Three kernels:
//  plan     (one block) checks the lengths and lists the pairs of tiles (2 TQ tokens) with the key blocks of 128 that
//           each sees, laid end to end for all key/value heads: a pair weighs its blocks and kPackedItemCost.
//  attend   (persistent) computes O = softmax(scale Q K^T + mask) V with an online softmax over the key blocks,
//           as in attention.cu: scores and O in TMEM, P in bf16 in the scores' columns.  Where that is even enough, the
//           CTAs are dealt whole pairs, heaviest first, back and forth.  Elsewhere (few long caches) the work is cut
//           into equal ranges, one for each group of CTAs (one CTA for each of up to 8 heads, which read neighbouring
//           cache rows at the same time); a range may begin and end inside a pair, at a block.  Whole / cut, us:
//           eight prompts of 11000 tokens 140 / 165, 16 heads of four prompts 89 / 104, 64 cached tokens 196 / 190.
//  combine  adds the parts of pairs that were cut: each left its unnormalised O, maximum and sum.
// Only keys of the sequence count: scores of rows past its end are masked by position and its last value
// tile is cleared past its end in shared memory, so whatever lies there (NaN included) has no effect.
//
// Bound: for prompts the tensor core and the exponentials, 1024 clocks each for a half block of 64 keys of two tiles, of which a
// 16384-token prompt with 32 and 8 heads reaches 0.85 (1300 - 1350 us, 1630 - 1690 TFLOP/s of the products that count); memory
// (K and V once per G heads) for single tokens: 64 over caches of up to 8064 keys in 190 us (0.89 of the copy rate).  A
// call's fixed part is about 13 us: the plan 5, the first loads and products of a CTA, its last output, the combination.
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
// The plan is a chain of short steps of one block: 512 threads take 0.8 us less than 1024, whose warps wait for issue slots.
constexpr int kPlanThreads = 512, kPlanWarps = kPlanThreads / 32;

// turn; per tile: Q, O free, drain; per ring slot: K, V; per tile and ring slot (2 x + slot): their releases; per tile and
// score buffer (2 x + buffer, which half blocks use in turn): S, P, P V done.  (Two P V may be outstanding when a
// softmax warp waits for the later one: with one barrier for both, its parity could not tell them apart.)
enum : int {
  B_Q_FULL = 0, B_Q_EMPTY = 2, B_K_FULL = 4, B_K_EMPTY = 6, B_V_FULL = 10, B_V_EMPTY = 12, B_S_FULL = 16,
  B_P_FULL = 20, B_PV_DONE = 24, B_O_FREE = 28, B_DRAIN = 30, B_TURN = 32, B_COUNT = 34
};

// ---- work list, in the workspace
struct PackedHeader {
  int64_t work, per;  // total weight; that of a group's range
  int pairs, whole;   // whole: pairs are not cut, and dealt out by weight
  int pad[58];
};
// A pair of tiles of one sequence, for every key/value head.
struct __align__(16) PackedPair {
  int q_row, qn;      // first query row; queries of the sequence from there on
  int k_row, klen;    // first key row, keys
  int pos0, eh;       // key position of query q_row; half blocks (64 keys) that the pair sees
  int64_t at;         // where it begins in the work (its head subgroups follow each other, eh + kPackedItemCost each)
};

// What cutting costs (parts' items, ranges that end at whole blocks, the combination), in half blocks: pairs stay
// whole where that leaves the longest share at most so much above the mean.
constexpr int kPackedCutCost = 16;
// What an item costs beside its half blocks (its first loads and products, its output), in half blocks: 2.5 us against
// 0.84 in eight ragged prompts.
constexpr int kPackedItemCost = 3;

__host__ __device__ inline int64_t up(int64_t n, int64_t a) { return (n + a - 1) / a * a; }

struct PackedLayout {
  int64_t starts, pairs, order, prefix, o, ml, total;
  int cap_pairs, slots;
};
constexpr int kSms = 152;  // CTAs that the workspace is sized for, at most
__host__ inline PackedLayout packed_layout(int64_t tq, int64_t n, int tokens, int64_t tk) {
  PackedLayout l;
  const bool cut = (tk + kBlk - 1) / kBlk >= 2 * kPackedMinPart;
  l.cap_pairs = static_cast<int>(tq / (2 * tokens) + n);  // of sequences that do not overlap
  l.slots = cut ? 4 * kSms : 0;                           // a CTA's first and last part, two tiles each
  l.starts = sizeof(PackedHeader);
  l.pairs = up(l.starts + kSms * 4, 256);
  l.order = up(l.pairs + int64_t(l.cap_pairs) * sizeof(PackedPair), 256);
  l.prefix = up(l.order + int64_t(l.cap_pairs) * 4, 256);
  l.o = up(l.prefix + (n > kPlanThreads ? n * 4 : 0), 1024);
  l.ml = l.o + int64_t(l.slots) * kBlk * kD * 4;
  l.total = l.ml + int64_t(l.slots) * 2 * kBlk * 4;
  return l;
}

struct PackedWork {
  PackedHeader* head;
  int* starts;         // the pair in which each group's range begins
  PackedPair* pairs;
  int* order;          // the pairs, heaviest first (where they are not cut)
  int* prefix;         // pairs before each sequence, where there are more sequences than threads
  float* o;            // slot: [column / 4][row][4]
  float* ml;           // slot: maximum (log2 domain) of the 128 rows, then their sums
  int cap_pairs;
};

// The block at which a range's border `off` into an item of eh half blocks cuts it: no part is shorter than
// kPackedMinPart (0 or all of its blocks: not cut).
__device__ __forceinline__ int cut_at(int64_t off, int eh) {
  const int e = (eh + 1) >> 1, b = off < eh ? static_cast<int>(off) >> 1 : e;
  return b < kPackedMinPart ? 0 : e - b < kPackedMinPart ? e : b;
}

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

// Half blocks of keys that the queries before tok1 of a sequence see.
__device__ __forceinline__ int seen_halves(int qlen, int klen, int tok1) {
  const int last = klen - qlen + min(tok1, qlen) - 1;
  return last < 0 ? 0 : (last >> 6) + 1;
}

template <class T>
__device__ __forceinline__ T block_scan(T v, T* warp_sums, T& total) {  // exclusive
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // the previous call's sums are read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    T s = lane < kPlanWarps ? warp_sums[lane] : T(0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xFFFFFFFFu, s, o);
      if (lane >= o) s += y;
    }
    if (lane < kPlanWarps) warp_sums[lane] = s;
  }
  __syncthreads();
  total = warp_sums[kPlanWarps - 1];
  return x - v + (warp > 0 ? warp_sums[warp - 1] : T(0));
}

__global__ void __launch_bounds__(kPlanThreads) packed_plan_kernel(const PackedArgs a, const PackedWork w) {
  __shared__ int sums[32];
  __shared__ long long sums64[32];
  __shared__ int near_prefix[kPlanThreads];
  __shared__ long long near_at[kPlanThreads];
  __shared__ int heaviest, longest, bins[kPlanThreads];
  __shared__ int4 near_seq[kPlanThreads];  // first query, queries, first key, keys
  const int tid = threadIdx.x, span = 2 * a.tokens;
  pdl_launch();
  if (tid == 0) heaviest = longest = 0;
  bins[tid] = 0;
  pdl_wait();
  // pairs of tiles before each sequence
  const bool near = a.n <= kPlanThreads;
  int64_t pairs64 = 0;
  for (int base = 0; base < a.n; base += kPlanThreads) {
    const int s = base + tid;
    int q0, qlen = 0, k0, klen;
    if (s < a.n) {
      seq_lengths(a, s, q0, qlen, k0, klen);
      if (near) near_seq[s] = make_int4(q0, qlen, k0, klen);
    }
    int total;
    const int before = block_scan((qlen + span - 1) / span, sums, total);
    if (s < a.n) (near ? near_prefix : w.prefix)[s] = static_cast<int>(pairs64) + before;
    pairs64 += total;
    if (pairs64 > w.cap_pairs) break;  // (uniform) overlapping sequences: refused below
  }
  __syncthreads();
  int pairs = static_cast<int>(pairs64);
  if (pairs64 > w.cap_pairs) {
    if (tid == 0) atomicCAS(&g_packed_err, 0, kPackedBadLengths);
    pairs = 0;
  }
  const int* prefix = near ? near_prefix : w.prefix;
  long long at = 0;
  int most = 0, first_eh = 0;
  for (int base = 0; base < pairs; base += kPlanThreads) {
    const int i = base + tid;
    PackedPair p = {};
    if (i < pairs) {
      int lo = 0, hi = a.n - 1;  // the last sequence that begins at or before pair i
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= i) lo = mid; else hi = mid - 1;
      }
      int q0, qlen, k0, klen;
      if (near) {
        const int4 v = near_seq[lo];
        q0 = v.x, qlen = v.y, k0 = v.z, klen = v.w;
      } else {
        seq_lengths(a, lo, q0, qlen, k0, klen);
      }
      const int tok0 = (i - prefix[lo]) * span;
      p.q_row = q0 + tok0;
      p.qn = qlen - tok0;
      p.k_row = k0;
      p.klen = klen;
      p.pos0 = klen - qlen + tok0;
      p.eh = seen_halves(qlen, klen, tok0 + span);
      most = max(most, p.eh);
      if (i == tid) first_eh = p.eh;
    }
    long long total;
    p.at = at + block_scan(i < pairs ? static_cast<long long>(p.eh + kPackedItemCost) * a.subgroups : 0ll, sums64, total);
    if (i < pairs) {
      w.pairs[i] = p;
      if (base == 0) near_at[tid] = p.at;
    }
    at += total;
  }
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  if ((tid & 31) == 0 && most > 0) atomicMax(&heaviest, most);
  __syncthreads();
  long long per = (at + a.groups - 1) / a.groups;
  if (per < 2 * kPackedMinPart + kPackedItemCost) per = 2 * kPackedMinPart + kPackedItemCost;
  // Whole pairs, dealt back and forth, where the longest of the CTAs' shares is near the mean (or, of many pairs, a
  // bound of it); a pair heavier than that decides it at once.
  const bool few = pairs <= kPlanThreads && a.hkv <= kPlanThreads;
  bool whole = few ? heaviest + kPackedItemCost <= per + kPackedCutCost
                   : 2ll * heaviest <= per && static_cast<long long>(pairs) * a.hkv < (1 << 30);
  if (whole) {
    // heaviest first: counting sort by half blocks (the order within a bin, of the threads' arrival, changes neither a
    // share nor a sum where a bin is one count)
    int shift = 0;
    while ((heaviest >> shift) >= kPlanThreads) ++shift;
    int* sorted = near_prefix;  // (read for the last time above)
    if (few && shift > 0) {
      // Bins of several counts would leave the shares below, and with them whether pairs are cut, to chance: each pair
      // counts those before it instead, the heavier and of equals the first.
      bins[tid] = first_eh;
      __syncthreads();
      if (tid < pairs) {
        int k = 0;
        for (int i = 0; i < pairs; ++i) k += bins[i] > first_eh || (bins[i] == first_eh && i < tid);
        w.order[k] = tid;
        sorted[k] = first_eh;
      }
      __syncthreads();
    } else {
      for (int i = tid; i < pairs; i += kPlanThreads)
        atomicAdd(&bins[kPlanThreads - 1 - ((i == tid ? first_eh : w.pairs[i].eh) >> shift)], 1);
      __syncthreads();
      int total;
      const int start = block_scan(bins[tid], sums, total);
      bins[tid] = start;
      __syncthreads();
      for (int i = tid; i < pairs; i += kPlanThreads) {
        const int eh = i == tid ? first_eh : w.pairs[i].eh, k = atomicAdd(&bins[kPlanThreads - 1 - (eh >> shift)], 1);
        w.order[k] = i;
        if (few) sorted[k] = eh;
      }
      __syncthreads();
    }
    if (few) {
      const int grid = a.groups * a.heads_abreast;
      const float per_head = 1.0f / static_cast<float>(a.hkv);
      int share = 0;
      if (tid < grid)
        for (int t = 0;; ++t) {
          const int i = t * grid + (t & 1 ? grid - 1 - tid : tid);
          const int k = static_cast<int>((static_cast<float>(i) + 0.5f) * per_head);  // i / hkv, exact below 2^21
          if (k >= pairs) break;
          share += sorted[k] + kPackedItemCost;
        }
      share = __reduce_max_sync(0xFFFFFFFFu, share);
      if ((tid & 31) == 0 && share > 0) atomicMax(&longest, share);
      __syncthreads();
      whole = longest <= per + kPackedCutCost;
    }
  }
  if (!whole && tid < a.groups) {
    const long long lo = tid * per;
    int first = 0, last = pairs - 1;
    while (first < last) {
      const int mid = (first + last + 1) >> 1;
      if ((pairs <= kPlanThreads ? near_at[mid] : w.pairs[mid].at) <= lo) first = mid; else last = mid - 1;
    }
    w.starts[tid] = first;
  }
  if (tid == 0) {
    w.head->work = at;
    w.head->per = per;
    w.head->pairs = pairs;
    w.head->whole = whole;
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

// As mbar_wait for a wait that may outlast any number of items: a tile that none of them uses waits for the next that
// does.  The bound grows with the CTA's share of the work (4 us a half block of 64 keys, which takes 0.8 or less).
__device__ __forceinline__ bool mbar_wait_share(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* err, int site,
                                                const PackedHeader* head) {
  uint64_t t0 = 0;
  for (uint32_t it = 0;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 63u) {
      if (*abort_flag) return false;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > kWaitTimeoutNs + 4000ull * static_cast<uint64_t>(head->per)) {
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

// This CTA's walk through the work: its group's range [lo, hi) in order, as items (pair, head subgroup); or, where
// pairs stay whole, items (pair, head) in the plan's order, dealt back and forth.
struct Walk {
  int pair, sub;           // next item (whole: pair is the round of dealing, sub -1)
  int cur_pair, cur_head;  // the one returned last

  __device__ Walk(const PackedArgs& a, const PackedWork& w) {
    pair = cur_pair = cur_head = 0;
    sub = -1;
    const int64_t lo = static_cast<int>(blockIdx.x) / a.heads_abreast * w.head->per;
    if (!w.head->whole && lo < w.head->work) {
      pair = w.starts[static_cast<int>(blockIdx.x) / a.heads_abreast];
      sub = static_cast<int>((lo - w.pairs[pair].at) / (w.pairs[pair].eh + kPackedItemCost));
    }
  }

  // Pair p of key head hk as far as it lies in the range; false if nothing of it does, with `end` if nothing after it does.
  __device__ bool item(const PackedArgs& a, const PackedWork& w, int p, int hk, Item& it, bool& end) const {
    const int4* entry = reinterpret_cast<const int4*>(w.pairs + p);
    const int4 u = entry[0], v = entry[1];
    const int eh = v.y, e = (eh + 1) >> 1, wide = eh + kPackedItemCost;
    const int64_t at = static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(v.z)) | (static_cast<uint64_t>(static_cast<uint32_t>(v.w)) << 32));
    // (the range: read again, rather than kept in registers)
    const int64_t lo = sub < 0 ? 0 : static_cast<int>(blockIdx.x) / a.heads_abreast * w.head->per;
    const int64_t hi = sub < 0 ? w.head->work : lo + w.head->per;
    const int64_t begin = at + static_cast<int64_t>(hk / a.heads_abreast) * wide;
    end = begin >= hi;
    if (end) return false;
    const int b0 = begin >= lo ? 0 : cut_at(lo - begin, eh), b1 = begin + wide <= hi ? e : cut_at(hi - begin, eh);
    if (b0 >= b1 && (e > 0 || begin < lo)) return false;  // (an item without blocks is its begin's)
    it.hk = hk;
    it.q_row = u.x;
    it.qn = u.y;
    it.k_row = u.z;
    it.klen = u.w;
    it.pos0 = v.x;
    it.b0 = b0;
    it.slot = b0 == 0 && b1 == e ? -1 : 4 * static_cast<int>(blockIdx.x) + (b0 > 0 ? 0 : 2);
    // the last position that each tile's queries see
    const int l0 = it.pos0 + min(a.tokens, it.qn) - 1, l1 = it.pos0 + min(2 * a.tokens, it.qn) - 1;
    it.e0 = min(2 * b1, l0 < 0 ? 0 : (l0 >> 6) + 1);
    it.e1 = it.qn > a.tokens ? min(2 * b1, l1 < 0 ? 0 : (l1 >> 6) + 1) : 0;
    it.last = (max(it.e0, it.e1) + 1) >> 1;
    if (it.last < it.b0) it.last = it.b0;
    return true;
  }

  __device__ bool next(const PackedArgs& a, const PackedWork& w, Item& it) {
    const int pairs = w.head->pairs;
    while (true) {
      if (sub < 0) {
        const int grid = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
        const int i = pair * grid + (pair & 1 ? grid - 1 - cta : cta);  // (the plan keeps this within 32 bits)
        ++pair;
        const int at = i / a.hkv;
        if (at >= pairs || !w.head->whole) return false;
        cur_head = i - at * a.hkv;
        cur_pair = w.order[at];
      } else {
        if (pair >= pairs) return false;
        cur_pair = pair;
        cur_head = sub * a.heads_abreast + static_cast<int>(blockIdx.x) % a.heads_abreast;
        if (++sub == a.subgroups) {
          sub = 0;
          ++pair;
        }
      }
      bool end;
      if (item(a, w, cur_pair, cur_head, it, end)) return true;
      if (end) return false;
    }
  }
};

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
      Walk walk(a, w);
      while (ok && walk.next(a, w, it)) {
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
      // each half block n P V of it and S of n + 2, in the same buffer.  The two issuers run freely, except that
      // tile 1's first scores of an item wait for tile 0's, which sets the tiles half a step apart (16384-token prompt
      // 1340 us; 1465 with the issuers taking turns throughout, 1355 with none; 8 ragged prompts 135, 139, 143).
      const uint32_t x = static_cast<uint32_t>(warp) - 1u;
      constexpr uint32_t kIdQK = idesc_bf16_f32(kBlk, 64, false, false);
      constexpr uint32_t kIdPV = idesc_bf16_f32(kBlk, kD, false, true);
      const uint64_t dQ = sdesc_sw128(sQ + x * kTile, 16, 1024), dK0 = sdesc_sw128(sK, 16, 1024),
                     dV0 = sdesc_sw128(sV, kHalf, 1024);
      const uint32_t tS = tmem_base + 128u * x, tO = tmem_base + 256u + 128u * x;
      const bool one = elect_one();
      uint32_t gb = 0, nq = 0, np = 0, turns = 0;  // ring position; items and half blocks of this tile; items of two tiles
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
      bool ok = true;
      auto k_ready = [&](int h) {
        const uint32_t r = gb + (static_cast<uint32_t>(h) >> 1);
        return mbar_wait(bar(B_K_FULL + (r & 1u)), (r >> 1) & 1u, abort_flag, err, a.err_site + 6);
      };
      Item it;
      Walk walk(a, w);
      while (ok && walk.next(a, w, it)) {
        const bool two = it.both();
        const int n = it.e(static_cast<int>(x)) - 2 * it.b0;  // half blocks of this tile
        const uint32_t blocks = static_cast<uint32_t>(it.last - it.b0);
        if (n > 0) {
          // after S of half block h: its block is released once its last half block of this tile is done
          auto made_s = [&](int h, uint32_t c) {
            umma_commit(bar(B_S_FULL + 2 * x + (c & 1u)));
            if ((h & 1) || h == n - 1) umma_commit(bar(B_K_EMPTY + 2 * x + ((gb + (static_cast<uint32_t>(h) >> 1)) & 1u)));
            if (h == n - 1) umma_commit(bar(B_Q_EMPTY + x));
          };
          if (!mbar_wait_share(bar(B_Q_FULL + x), nq & 1u, abort_flag, err, a.err_site + 5, w.head) || !k_ready(0) ||
              (two && x == 1 && !mbar_wait(bar(B_TURN + (turns & 1u)), (turns >> 1) & 1u, abort_flag, err, a.err_site + 4))) {
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
            // (tile 0 may be a whole item ahead, not two: the rings hold two blocks; hence two barriers)
            if (two && x == 0) mbar_arrive(bar(B_TURN + (turns & 1u)));
          }
          if (two) ++turns;
          for (int h = 0; ok && h < n; ++h) {
            const uint32_t r = gb + (static_cast<uint32_t>(h) >> 1);
            // the waits that are usually over first, the softmax hand-off (the critical path) last
            if (!mbar_wait(bar(B_V_FULL + (r & 1u)), (r >> 1) & 1u, abort_flag, err, a.err_site + 7) ||
                (h + 2 < n && !k_ready(h + 2)) ||
                // the item's first P V overwrites O: the previous item's must be read
                (h == 0 && nq > 0 && !mbar_wait(bar(B_O_FREE + x), (nq - 1) & 1u, abort_flag, err, a.err_site + 8)) ||
                !mbar_poll(bar(B_P_FULL + 2 * x + (np & 1u)), (np >> 1) & 1u, abort_flag, err, a.err_site + 9)) {
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
            }
            ++np;
          }
          ++nq;
        }
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
    Walk walk(a, w);
    while (ok && walk.next(a, w, it)) {
      const int e = it.e(x), first = 2 * it.b0, klen = it.klen;
      // the last key position that this row sees (none for rows outside)
      const int lim = row < rows && tok < it.qn - x * a.tokens ? min(it.pos0 + x * a.tokens + tok, klen - 1) : -1;
      float m_run = -INFINITY, l_run = 0.0f;
      for (int j = first; ok && j < e; ++j, ++cb) {
        const uint32_t tB = tS + 64u * (cb & 1u);
        ok = mbar_wait_share(bar(B_S_FULL + 2 * x + (cb & 1u)), (cb >> 1) & 1u, abort_flag, err, a.err_site + 10, w.head);
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
        // The running maximum is raised when some row of the warp would pass it by more than 8 in the log2 domain
        // (p <= 2^8 otherwise); O and the sum are then rescaled.  A row that has seen no key keeps -inf, and zero
        // stands in for it so that its p are 0 and not NaN.  Where the maximum's product with the scale has no binary
        // places left (2^28), its rounding would be off by more than 2^ can take; scores that differ are then so far
        // apart that one key has all the weight at any scale, and a power of two, which rounds nothing, stands in.
        const float cand = fmaxf(m_run, top);
        const bool raise = __any_sync(0xFFFFFFFFu, cand - m_run > a.raise_by) || j == first;
        const float mx = raise ? cand : m_run;
        const float sc = fabsf(mx) < a.huge ? a.scale_log2 : a.scale_two;
        const float base = mx == -INFINITY ? 0.0f : __fmul_rn(mx, sc);
        const float alpha = raise ? ex2_approx(__fmul_rn(m_run, sc) - base) : 1.0f;
        uint64_t l4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) l4[i] = f2(0.0f, 0.0f);
        const uint64_t sc2 = f2(sc, sc), nmx2 = f2(-base, -base);
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
      bool end;
      walk.item(a, w, walk.cur_pair, walk.cur_head, it, end);  // again, rather than kept in registers through the blocks
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
          ml[row] = m_run * a.scale_log2;
          ml[kBlk + row] = l_run;
        }
        continue;
      }
      // O / sum -> bf16, 64 columns at a time through this warp's box (32 rows x 128 bytes, 16-byte piece
      // j of row r at j ^ (r % 8)), then row by row with eight lanes each; rows without keys are zero
      const float inv = l_run > 0.0f || l_run != l_run ? 1.0f / l_run : 0.0f;
      if (row_ok && a.lse)
        a.lse[static_cast<int64_t>(it.q_row + x * a.tokens + tok) * a.hq + it.hk * a.group + (row - tok * a.group)] =
            l_run > 0.0f || l_run != l_run ? (__fmul_rn(m_run, a.scale_log2) + log2f(l_run)) * 0.69314718055994531f : -INFINITY;
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
// Block (border, head of the group, tile and a quarter of O's columns), for the first border that cuts an item: with
// m = max m_p and c_p = 2^(m_p - m) over the item's parts p in order, O = sum c_p O_p / sum c_p l_p, lse = ln 2 (m + log2(sum c_p l_p)).
__global__ void __launch_bounds__(256) packed_combine_kernel(const PackedArgs a, const PackedWork w) {
  pdl_launch();
  pdl_wait();
  const int g = static_cast<int>(blockIdx.x) + 1, j = blockIdx.y, x = blockIdx.z & 1, quarter = blockIdx.z >> 1;
  const int64_t per = w.head->per;
  if (g * per >= w.head->work || w.head->whole) return;
  const PackedPair p = w.pairs[w.starts[g]];
  const int blocks = (p.eh + 1) >> 1, wide = p.eh + kPackedItemCost, sub = static_cast<int>((g * per - p.at) / wide);
  const int64_t begin = p.at + static_cast<int64_t>(sub) * wide;
  auto border = [&](int k) { return k * per <= begin ? 0 : cut_at(k * per - begin, p.eh); };  // where border k cuts the item
  const int b = border(g), before = border(g - 1);
  if (b == 0 || b == blocks || before > 0) return;  // not cut here, or already before
  const int live = min(a.tokens, p.qn - x * a.tokens);
  if (live <= 0) return;
  const int last = p.pos0 + x * a.tokens + live - 1, e = last < 0 ? 0 : (last >> 7) + 1;
  // parts that hold some of the tile's blocks: the first is group g - 1's last, the k-th after it group (g - 1 + k)'s first
  int parts = e > 0 ? 1 : 0;
  while (parts > 0 && border(g - 1 + parts) < e) ++parts;
  const int hk = sub * a.heads_abreast + j, rows = live * a.group;
  auto slot = [&](int k) { return static_cast<int64_t>(4 * ((g - 1 + k) * a.heads_abreast + j) + (k == 0 ? 2 : 0) + x); };
  for (int i = threadIdx.x; i < rows * 8; i += 256) {
    const int row = i % rows, c = quarter * 8 + i / rows;  // piece c: columns 4 c .. 4 c + 3
    float m = -INFINITY;
#pragma unroll 8
    for (int k = 0; k < parts; ++k) m = fmaxf(m, w.ml[slot(k) * (2 * kBlk) + row]);
    float l = 0.0f, o0 = 0.0f, o1 = 0.0f, o2 = 0.0f, o3 = 0.0f;
    const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll 4
    for (int k = 0; k < parts; ++k) {
      const float* ml = w.ml + slot(k) * (2 * kBlk);
      const float f = exp2f(ml[row] - base);
      const float4 v = *reinterpret_cast<const float4*>(w.o + slot(k) * (kBlk * kD) + (c * kBlk + row) * 4);
      l = fmaf(f, ml[kBlk + row], l);
      o0 = fmaf(f, v.x, o0);
      o1 = fmaf(f, v.y, o1);
      o2 = fmaf(f, v.z, o2);
      o3 = fmaf(f, v.w, o3);
    }
    const bool some = l > 0.0f || l != l;
    const float inv = some ? 1.0f / l : 0.0f;
    const int t = row / a.group;
    const int64_t token = p.q_row + x * a.tokens + t;
    const int head = hk * a.group + row - t * a.group;
    *reinterpret_cast<uint2*>(a.O + token * a.ld_o + static_cast<int64_t>(head) * kD + c * 4) =
        make_uint2(pack_bf16x2(o0 * inv, o1 * inv), pack_bf16x2(o2 * inv, o3 * inv));
    if (c == 0 && a.lse) a.lse[token * a.hq + head] = some ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
  }
}

PackedWork packed_work(const PackedArgs& a, void* ws) {
  const PackedLayout l = packed_layout(a.tq, a.n, a.tokens, a.tk);
  uint8_t* p = static_cast<uint8_t*>(ws);
  PackedWork w;
  w.head = reinterpret_cast<PackedHeader*>(p);
  w.starts = reinterpret_cast<int*>(p + l.starts);
  w.pairs = reinterpret_cast<PackedPair*>(p + l.pairs);
  w.order = reinterpret_cast<int*>(p + l.order);
  w.prefix = reinterpret_cast<int*>(p + l.prefix);
  w.o = reinterpret_cast<float*>(p + l.o);
  w.ml = reinterpret_cast<float*>(p + l.ml);
  w.cap_pairs = l.cap_pairs;
  return w;
}

}  // namespace

int64_t packed_scratch_bytes(int64_t tq, int64_t n, int hq, int hkv, int64_t tk) {
  return packed_layout(tq, n, kBlk / (hq / hkv), tk).total;
}

void packed_groups(PackedArgs* a, int sms) {
  // the largest divisor of the key heads up to 8; at most 7 CTAs of a GPU stay idle for it
  a->heads_abreast = 8;
  while (a->hkv % a->heads_abreast != 0) --a->heads_abreast;
  a->subgroups = a->hkv / a->heads_abreast;
  a->groups = (sms < kSms ? sms : kSms) / a->heads_abreast;
  if (a->groups < 1) a->groups = 1;
}

cudaError_t launch_packed_plan(const PackedArgs& a, void* ws, cudaStream_t st) {
  return launch_pdl(packed_plan_kernel, dim3(1), dim3(kPlanThreads), 0, 1, st, a, packed_work(a, ws));
}

cudaError_t launch_packed_attention(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                                    const PackedArgs& a, void* ws, cudaStream_t st) {
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
  return launch_pdl(packed_attention_kernel, dim3(static_cast<unsigned>(a.groups * a.heads_abreast)), dim3(kThreads), kSmem, 1, st, q,
                    k, v, a, packed_work(a, ws));
}

bool packed_may_cut(const PackedArgs& a) { return a.groups > 1 && packed_layout(a.tq, a.n, a.tokens, a.tk).slots > 0; }

cudaError_t launch_packed_combine(const PackedArgs& a, void* ws, cudaStream_t st) {
  return launch_pdl(packed_combine_kernel, dim3(static_cast<unsigned>(a.groups - 1), static_cast<unsigned>(a.heads_abreast), 8), dim3(256),
                    0, 1, st, a, packed_work(a, ws));
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
