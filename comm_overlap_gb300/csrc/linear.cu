// linear.cu -- the linear layer's products: D = A . B^T (bf16 operands, either one contiguous along
// the reduction or along its rows, fp32 accumulation) with an epilogue that adds a bias, keeps the
// pre-activation, applies an activation, adds a residual and rounds once to bf16; and the column
// pass of the backward (gZ = gY act'(Z), bias gradient).
//
// The product runs on CTA pairs (tcgen05.mma.cta_group::2, tiles of 256 rows and `width` columns, 64
// elements of the reduction a step through a TMA ring of five stages or more):
//   warp 0 (an elected lane)  TMA producer of this CTA's 128 rows of A and its width / 2 rows of B
//   warp 1 (an elected lane of the leader)  MMA issuer, two 256-column accumulators in TMEM
//   warps 2-9          epilogue, two per TMEM lane quarter taking alternate 32-column chunks, one row a
//                      thread
// The launcher lays the work over the GPU (lin_plan): pairs take tiles unit, unit + units, ...; the width
// (64 to 256 columns) is chosen so that the last round leaves few pairs idle; a product with few tiles is
// also cut along the reduction over the 2 or 4 pairs of a larger cluster, whose fp32 partials meet in
// shared memory and are added in their order, each pair finishing a part of the rows.  No sum's
// order depends on timing.
//
// Bound: the tensor core.  16384 x 16384 -> 4096 takes 1140 - 1250 us (0.91 - 1.0 of the measured burst rate; the power
// cap decides), 777 x 2560 -> 10240 with GeLU and its pre-activation 39 us (21 at the burst rate): its last tile of
// rows is nearly all padding, and every step is bound by staging its operands (lin_plan).
#include "gelu2.cuh"
#include "gemm.cuh"
#include "ops.h"

namespace dm {

namespace {

constexpr int kLinThreads = 320;
constexpr int kLinRing = 5 * 32768;  // the operand ring: stages of 64 elements of a_rows rows of A and the B rows
constexpr int kLinMaxStages = 16;    // as many as fit, at least 5 (128 rows of A and of B)
constexpr int kLinBox = 2048;          // 32 x 32 bf16
constexpr int kLinWarpBytes = 4 * kLinBox;  // an epilogue warp's boxes: a Y for each of its chunks, or two Y and Z
constexpr int kLinSmem = 1024 + kCtrlBytes + kLinRing + 8 * kLinWarpBytes;
static_assert(kLinSmem <= 232448, "shared memory beyond the per-CTA limit");
static_assert(128 * 256 * 4 <= kLinRing, "a partial fits the idle ring");

// Tiles in groups of 8 rows of tiles, so that the operands of concurrent tiles stay in L2.
__device__ __forceinline__ void lin_tile(const LinArgs& a, int tile, int& mt, int& nt) {
  const int span = kGroupM * a.n_tiles;
  const int grp = tile / span, first = grp * kGroupM, size = min(a.m_tiles - first, kGroupM), in = tile - grp * span;
  mt = first + in % size;
  nt = in / size;
}

__device__ __forceinline__ void st_shared_cluster_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// drain_pair_ring (gemm.cuh) for a ring of `stages` stages.
__device__ __forceinline__ void drain_ring(uint32_t full_bar0, uint32_t stages, uint32_t own, uint32_t peer,
                                           uint32_t peer_bytes) {
  const uint32_t end = own > peer ? own : peer;
#pragma unroll 1
  for (uint32_t s = 0; s < stages && s < end; ++s) {
    const uint32_t j = s + (end - 1u - s) / stages * stages;  // last use of stage s below `end`
    if (j < own && j >= peer)
      mbar_complete_tx(full_bar0 + 8u * s, peer_bytes);
    else if (j >= own && j < peer)
      mbar_arrive_expect_tx(full_bar0 + 8u * s, peer_bytes);
    mbar_wait_drain(full_bar0 + 8u * s, (j / stages) & 1u);
  }
}

// Bound of the wait for a whole accumulator: the time of its steps (0.1 - 0.4 us each) comes on top of that for one step.
__device__ __forceinline__ uint64_t acc_wait_ns(int steps) { return kWaitTimeoutNs + 4000ull * static_cast<uint64_t>(steps); }

// Bias and residual of a 32-column chunk (first column col) for one row; zero outside D.
struct LinIn {
  uint4 bias[4], res[4];
  __device__ __forceinline__ void load(const LinArgs& a, int row, int col) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool in = col + 8 * q < a.N;
      bias[q] = in && a.bias ? *reinterpret_cast<const uint4*>(a.bias + col + 8 * q) : make_uint4(0u, 0u, 0u, 0u);
      res[q] = in && a.R && row < a.M
                   ? *reinterpret_cast<const uint4*>(a.R + static_cast<int64_t>(row) * a.ld_r + col + 8 * q)
                   : make_uint4(0u, 0u, 0u, 0u);
    }
  }
};

// Epilogue of one 32-column chunk (first column col) of the rows row0 + lane, r: the sums.
__device__ __forceinline__ void lin_chunk(const LinArgs& a, const CUtensorMap* tmY, const CUtensorMap* tmZ,
                                          const uint32_t (&r)[32], const LinIn& in, int row0, int col, int lane,
                                          uint32_t boxes, uint32_t& n_stored) {
  // Z = D + bias; Y = act(Z) + R, each rounded once from fp32
  uint32_t y[16], z[16];
  auto finish = [&](auto act) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t bw[4] = {in.bias[q].x, in.bias[q].y, in.bias[q].z, in.bias[q].w};
      const uint32_t rw[4] = {in.res[q].x, in.res[q].y, in.res[q].z, in.res[q].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float z0 = __uint_as_float(r[8 * q + 2 * e]) + bf16lo(bw[e]);
        const float z1 = __uint_as_float(r[8 * q + 2 * e + 1]) + bf16hi(bw[e]);
        z[4 * q + e] = pack_bf16x2(z0, z1);
        float y0, y1;
        if constexpr (decltype(act)::value == ACT_GELU) {
          gelu_f2(z0, z1, y0, y1);
        } else if constexpr (decltype(act)::value == ACT_RELU) {
          y0 = max_nan(z0, 0.0f);
          y1 = max_nan(z1, 0.0f);
        } else {
          y0 = z0;
          y1 = z1;
        }
        y[4 * q + e] = pack_bf16x2(y0 + bf16lo(rw[e]), y1 + bf16hi(rw[e]));
      }
    }
  };
  if (a.act == ACT_GELU)
    finish(std::integral_constant<int, ACT_GELU>{});
  else if (a.act == ACT_RELU)
    finish(std::integral_constant<int, ACT_RELU>{});
  else
    finish(std::integral_constant<int, ACT_NONE>{});
  // the boxes in turn (32 x 64 bytes, 16-byte piece j of row r at j ^ (r / 2 % 4)): four Y, or two pairs
  const uint32_t box = boxes + (a.save ? (n_stored & 1u) * 2u : (n_stored & 3u)) * kLinBox;
  if (lane == 0) {
    if (a.save) bulk_wait_group_read<1>();
    else bulk_wait_group_read<3>();
  }
  __syncwarp();
  const uint32_t at = box + static_cast<uint32_t>(lane) * 64u, x = (static_cast<uint32_t>(lane) >> 1) & 3u;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t off = (static_cast<uint32_t>(j) ^ x) << 4;
    st_shared_v4(at + off, y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
    if (a.save) st_shared_v4(at + kLinBox + off, z[4 * j], z[4 * j + 1], z[4 * j + 2], z[4 * j + 3]);
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_3d(tmY, box, col, row0, 0);
    if (a.save) tma_store_3d(tmZ, box + kLinBox, col, row0, 0);
    bulk_commit_group();
  }
  ++n_stored;
}

// Output column n of rows m0 and m1 (none if negative) from the sums with bias z and the residuals r.
__device__ __forceinline__ void few_put(const LinFewArgs& a, int n, bool live, int m0, int m1, float z0, float z1, float r0, float r1) {
  float y0 = z0, y1 = z1;
  if (a.act == ACT_GELU) {
    gelu_f2(z0, z1, y0, y1);
  } else if (a.act == ACT_RELU) {
    y0 = max_nan(z0, 0.0f);
    y1 = max_nan(z1, 0.0f);
  }
  if (!live) return;
  const uint32_t y = pack_bf16x2(y0 + r0, y1 + r1), z = pack_bf16x2(z0, z1);
  a.Y[m0 * a.ld_y + n] = static_cast<uint16_t>(y);
  if (a.Z) a.Z[m0 * a.ld_z + n] = static_cast<uint16_t>(z);
  if (m1 < 0) return;
  a.Y[m1 * a.ld_y + n] = static_cast<uint16_t>(y >> 16);
  if (a.Z) a.Z[m1 * a.ld_z + n] = static_cast<uint16_t>(z >> 16);
}

template <bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmZ, const LinArgs a) {
  constexpr int S = kLinMaxStages;
  constexpr int kFull = 0, kEmpty = S, kAccFull = 2 * S, kAccEmpty = 2 * S + 2, kDrain = 2 * S + 4,
                kPeerCount = 2 * S + 5;
  static_assert(8 * (kPeerCount + 1) <= 512, "barriers overlap the TMEM slot");
  const uint32_t stages = static_cast<uint32_t>(a.stages), stage_bytes = static_cast<uint32_t>(a.stage_bytes),
                 b_at = static_cast<uint32_t>(a.a_rows) * 128u;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + 512);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + 516);
  volatile uint32_t* peer_issued = reinterpret_cast<volatile uint32_t*>(smem + 520);
  const uint32_t bar0 = smem_u32(smem), stage0 = smem_u32(smem + kCtrlBytes);
  auto bar = [bar0](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // CTA `crank` of the cluster: half `rank` of pair `part`, which computes part `part` of the reduction
  const uint32_t crank = cluster_ctarank(), rank = crank & 1u, lead = crank & ~1u;
  const int part = static_cast<int>(crank >> 1);
  const bool leader = rank == 0;
  const int unit = static_cast<int>(blockIdx.x) / (2 * a.parts), units = static_cast<int>(gridDim.x) / (2 * a.parts);
  const uint16_t pair_mask = static_cast<uint16_t>(3u << lead);
  const int k_first = part * a.k_blocks / a.parts, k_last = (part + 1) * a.k_blocks / a.parts;
  const int tiles = a.m_tiles * a.n_tiles;
  int* err = &g_gemm_err;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(bar(kFull + s), 1);
      mbar_init(bar(kEmpty + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kAccFull + i), 1);
      mbar_init(bar(kAccEmpty + i), 16);  // eight epilogue warps of each CTA
    }
    mbar_init(bar(kDrain), 1);
    mbar_init(bar(kPeerCount), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&tmA);
    tma_prefetch_map(&tmB);
    tma_prefetch_map(&tmY);
    if (a.save) tma_prefetch_map(&tmZ);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  pdl_launch();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();

  if (warp == 0) {
    {
      // ---------------- TMA producer (the warp walks the loop, one elected lane issues)
      const bool one = elect_one();
      uint32_t s = 0, ph = 0, issued = 0;
      bool ok = true;
      const uint32_t full_lead = mapa_shared(bar(kFull), lead);
      const uint32_t b_rows = static_cast<uint32_t>(a.width) / 2;
      const uint32_t b_bytes = (B_MN ? (b_rows + 63u) / 64u * 64u : b_rows) * 128u;
      // with at most 128 rows of A the second CTA has none: it loads none, and its accumulator is not read
      const bool has_a = leader || a.M > 128;
      const uint32_t a_bytes = static_cast<uint32_t>(a.a_rows) * 128u;
      const uint32_t peer_bytes = (a.M > 128 ? a_bytes : 0u) + b_bytes;
      for (int tile = unit; ok && tile < tiles; tile += units) {
        int mt, nt;
        lin_tile(a, tile, mt, nt);
        const int m0 = mt * 256 + static_cast<int>(rank) * 128, n0 = nt * a.width + static_cast<int>(rank * b_rows);
        for (int kb = k_first; kb < k_last; ++kb) {
          ok = mbar_wait(bar(kEmpty + s), ph ^ 1u, abort_flag, err, a.err_site + 1);
          if (!ok) break;
          const uint32_t sa = stage0 + s * stage_bytes, sb = sa + b_at;
          const uint32_t fb = full_lead + 8u * s;  // the leader's barrier counts both CTAs' bytes
          const int k0 = kb * kBK;
          if (one) {
          if (leader) mbar_arrive_expect_tx(bar(kFull + s), a_bytes + b_bytes + peer_bytes);
          if (has_a) {
            if constexpr (!A_MN) {
              tma_load_3d_pair(sa, &tmA, fb, k0, m0, 0);
            } else {
              tma_load_3d_pair(sa, &tmA, fb, m0, k0, 0);
              tma_load_3d_pair(sa + 8192, &tmA, fb, m0 + 64, k0, 0);
            }
          }
          if constexpr (!B_MN) {
            tma_load_3d_pair(sb, &tmB, fb, k0, n0, 0);
          } else {
            tma_load_3d_pair(sb, &tmB, fb, n0, k0, 0);
            if (b_rows > 64) tma_load_3d_pair(sb + 8192, &tmB, fb, n0 + 64, k0, 0);
          }
          }
          ++issued;
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // both CTAs' copies have landed before the pair leaves, also after an abort (gemm.cuh)
      if (!one) {
      } else if (!leader) {
        st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t*>(peer_issued)), lead), issued);
        mbar_arrive_cluster(mapa_shared(bar(kPeerCount), lead));
      } else if (mbar_wait_cluster_acquire(bar(kPeerCount), 0, kPeerCountTimeoutNs)) {
        const uint32_t peer = *peer_issued;
        if (!ok || peer != issued || *abort_flag) drain_ring(bar(kFull), stages, issued, peer, peer_bytes);
      } else {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < kPeerCopyGraceNs) {
        }
      }
    }
    __syncwarp();
    if (a.parts > 1) {  // the epilogue's two
      cluster_sync();
      cluster_sync();
    }
  } else if (warp == 1) {
    if (leader) {
      // ---------------- MMA issuer for both CTAs.  The whole warp walks the loop and one elected lane issues:
      // the operands are then warp-uniform, and a product's issue costs a fraction of what it costs a thread of
      // a diverged warp (measured: 134 clocks, as long as a 256 x 256 x 16 product takes).
      const bool one = elect_one();
      uint32_t s = 0, ph = 0;
      bool ok = true;
      const uint32_t idesc = idesc_bf16_f32(256, a.width, A_MN, B_MN);
      const uint64_t a_desc = A_MN ? sdesc_sw128(stage0, 8192, 1024) : sdesc_sw128(stage0, 16, 1024);
      const uint64_t b_desc = B_MN ? sdesc_sw128(stage0 + b_at, 8192, 1024) : sdesc_sw128(stage0 + b_at, 16, 1024);
      int i = 0;
      for (int tile = unit; ok && tile < tiles; tile += units, ++i) {
        const int acc = i & 1;
        ok = mbar_wait(bar(kAccEmpty + acc), ((static_cast<uint32_t>(i) >> 1) & 1u) ^ 1u, abort_flag, err,
                       a.err_site + 2);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kBN);
        for (int kb = k_first; kb < k_last; ++kb) {
          ok = mbar_wait(bar(kFull + s), ph, abort_flag, err, a.err_site + 3);
          if (!ok) break;
          tc_fence_after();
          const uint64_t off = static_cast<uint64_t>(s * stage_bytes >> 4);
          if (one) {
#pragma unroll
            for (int kk = 0; kk < kBK / 16; ++kk)
              umma_bf16_pair(d, a_desc + off + (A_MN ? kk * 128 : kk * 2), b_desc + off + (B_MN ? kk * 128 : kk * 2), idesc,
                             static_cast<uint32_t>(kb != k_first || kk != 0));
            umma_commit_pair_multicast(bar(kEmpty + s), pair_mask);
          }
          if (++s == stages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        if (one) umma_commit_pair_multicast(bar(kAccFull + acc), pair_mask);
      }
      if (one) umma_commit_pair(bar(kDrain));
      __syncwarp();
      mbar_wait_drain(bar(kDrain), 0);
    }
    __syncwarp();
    if (a.parts > 1) {  // the epilogue's two
      cluster_sync();
      cluster_sync();
    }
  } else {
    // ---------------- epilogue: rows of the warp's TMEM lane quarter, every other 32-column chunk
    const int ew = warp - 2, quarter = warp & 3, half = ew >> 2;
    const uint32_t boxes = stage0 + kLinRing + static_cast<uint32_t>(ew) * kLinWarpBytes;
    const uint32_t tq = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16);
    uint32_t n_stored = 0;
    if (a.parts == 1) {
      int i = 0;
      for (int tile = unit; tile < tiles; tile += units, ++i) {
        int mt, nt;
        lin_tile(a, tile, mt, nt);
        const int row0 = mt * 256 + static_cast<int>(rank) * 128 + quarter * 32;
        const int acc = i & 1;
        // a chunk's bias and residual are loaded before the previous one is finished (the first's while the
        // products run)
        LinIn in;
        in.load(a, row0 + lane, nt * a.width + 32 * half);
        const bool ok = mbar_wait(bar(kAccFull + acc), (static_cast<uint32_t>(i) >> 1) & 1u, abort_flag, err, a.err_site + 4,
                                  acc_wait_ns(k_last - k_first));
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        tc_fence_after();
        const uint32_t tacc = tq + static_cast<uint32_t>(acc * kBN);
#pragma unroll 1
        for (int cc = 32 * half; cc < a.width; cc += 64) {
          const int col = nt * a.width + cc;
          if (row0 >= a.M || col >= a.N) break;
          uint32_t r[32];
          tmem_ld32(tacc + static_cast<uint32_t>(cc), r);
          const LinIn now = in;
          if (cc + 64 < a.width) in.load(a, row0 + lane, col + 64);
          tmem_ld_wait();
          lin_chunk(a, &tmY, &tmZ, r, now, row0, col, lane, boxes, n_stored);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(bar(kAccEmpty + acc), lead));
      }
    } else {
      // one tile a cluster: each pair sends its fp32 partial of lane quarter qd to the pair that finishes it,
      // qd / (4 / parts), into that CTA's ring, block `part` (4 / parts x 32 rows, 16-byte piece j of row r
      // at j ^ (r % 8)); the finishing pair adds the blocks in their order
      int mt, nt;
      lin_tile(a, unit, mt, nt);
      const int row_cta = mt * 256 + static_cast<int>(rank) * 128, rows4 = 4 / a.parts;
      const uint32_t row_bytes = static_cast<uint32_t>(a.width) * 4u, key = static_cast<uint32_t>(lane) & 7u;
      const uint32_t block = static_cast<uint32_t>(rows4) * 32u * row_bytes;
      const bool got = mbar_wait(bar(kAccFull), 0, abort_flag, err, a.err_site + 4, acc_wait_ns(k_last - k_first));
      const bool ok = __all_sync(0xFFFFFFFFu, got);
      tc_fence_after();
      cluster_sync();  // every ring of the cluster is idle (after an abort: nothing is sent or read)
      if (ok && row_cta + quarter * 32 < a.M) {
        const uint32_t p = mapa_shared(stage0, static_cast<uint32_t>(quarter / rows4 * 2) + rank) + static_cast<uint32_t>(part) * block +
                           static_cast<uint32_t>(quarter % rows4 * 32 + lane) * row_bytes;
#pragma unroll 1
        for (int cc = 32 * half; cc < a.width; cc += 64) {
          uint32_t r[32];
          tmem_ld32(tq + static_cast<uint32_t>(cc), r);
          tmem_ld_wait();
          if (row_cta + quarter * 32 + lane < a.M) {
#pragma unroll
            for (uint32_t j = 0; j < 8; ++j)
              st_shared_cluster_v4(p + (((static_cast<uint32_t>(cc) / 4u + j) ^ key) << 4), r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      cluster_sync();  // every block has arrived
      if (ok) {
        const int chunks = a.width / 32;
#pragma unroll 1
        for (int c = ew; c < rows4 * chunks; c += 8) {
          const int qd = c / chunks, cc = (c - qd * chunks) * 32;
          const int row0 = row_cta + (part * rows4 + qd) * 32, col = nt * a.width + cc;
          if (row0 >= a.M || col >= a.N) continue;
          const uint32_t p = stage0 + static_cast<uint32_t>(qd * 32 + lane) * row_bytes;
          uint32_t r[32];
          LinIn in;
          in.load(a, row0 + lane, col);
#pragma unroll 1
          for (int q = 0; q < a.parts; ++q) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint4 v = ld_shared_v4(p + static_cast<uint32_t>(q) * block +
                                           (((static_cast<uint32_t>(cc) / 4u + static_cast<uint32_t>(j)) ^ key) << 4));
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                r[4 * j + e] = q == 0 ? w[e] : __float_as_uint(__uint_as_float(r[4 * j + e]) + __uint_as_float(w[e]));
            }
          }
          lin_chunk(a, &tmY, &tmZ, r, in, row0, col, lane, boxes, n_stored);
        }
      }
    }
    if (lane == 0) bulk_wait_group_all();
    __syncwarp();
  }

  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

template <bool A_MN, bool B_MN>
cudaError_t launch_linear_t(const LinMaps& m, const LinArgs& a, cudaStream_t st) {
  auto fn = linear_kernel<A_MN, B_MN>;
  static std::atomic<bool> ready_of[kMaxDevices];  // the shared-memory opt-in, per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!ready_of[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kLinSmem);
    if (e != cudaSuccess) return e;
    ready_of[dev].store(true, std::memory_order_release);
  }
  return launch_pdl(fn, dim3(static_cast<unsigned>(2 * a.parts * a.units)), dim3(kLinThreads), kLinSmem, 2 * a.parts, st,
                    m.a, m.b, m.y, m.z, a);
}

// ---- The layer on few rows: bound by the bytes of W, which every SM streams through its own tensor core.  W takes the
// place of the wide operand (a tile is `height` <= 128 of its rows; the product's other lanes read what lies behind
// them in the ring and are not used), X that of the narrow one (M rounded up to 16), so that a step costs shared
// memory little more than W itself, and an output column is a lane: the epilogue is one column a thread, for all
// rows of X.  Where N gives too few tiles, the CTAs of a cluster split the reduction and send their sums to the one
// that finishes a row (row m by CTA m % parts), which adds them in the CTAs' order.  A stage is two swizzle panels,
// 256 contiguous bytes of each row of W: with one panel 16384 x 4096 takes 23.1 us instead of 22.2 for one row and
// 8192 x 8192 27.4 instead of 23.4.  The kernel for many rows takes 27.1 us for one row of 16384 x 4096 with GeLU
// (this one 22.2; W at the copy rate 19.8), 28.3 for 64 rows (25.6); 28.4 and 31.3 for 4096 x 16384 (23.5, 30.4).
constexpr int kFewPanels = 2;  // of 64 elements of the reduction a stage
constexpr int kFewStages = 24, kFewRing = 196608, kFewJoin = kFewRows * 128 * 4;
constexpr int kFewSmem = 1024 + kCtrlBytes + kFewRing + kFewJoin;
static_assert(kFewSmem <= 232448, "shared memory beyond the per-CTA limit");
static_assert(kFewJoin >= 128 * 128, "the last stage's unused lanes read past the ring");

__device__ __forceinline__ void st_shared_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__global__ void __launch_bounds__(kLinThreads, 1)
    linear_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const LinFewArgs a) {
  constexpr int S = kFewStages, kFull = 0, kEmpty = S, kAccFull = 2 * S, kAccEmpty = 2 * S + 2, kDrain = 2 * S + 4;
  static_assert(8 * (kDrain + 1) <= 512, "barriers overlap the TMEM slot");
  static_assert(2 * kFewRows <= 128, "two accumulators");
  constexpr uint32_t kCols = 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + 512);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + 516);
  const uint32_t bar0 = smem_u32(smem), stage0 = smem_u32(smem + kCtrlBytes), join = stage0 + kFewRing;
  auto bar = [bar0](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  const uint32_t stages = static_cast<uint32_t>(a.stages), stage_bytes = static_cast<uint32_t>(a.stage_bytes),
                 w_panel = static_cast<uint32_t>(a.height) * 128u, x_panel = static_cast<uint32_t>(a.x_rows) * 128u,
                 x_at = kFewPanels * w_panel;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = static_cast<int>(cluster_ctarank());
  const int unit = static_cast<int>(blockIdx.x) / a.parts, units = static_cast<int>(gridDim.x) / a.parts;
  const int k_first = part * a.k_blocks / a.parts, k_last = (part + 1) * a.k_blocks / a.parts;
  int* err = &g_gemm_err;

  if (threadIdx.x == 0) {
    for (int i = 0; i <= kDrain; ++i) mbar_init(bar(i), i >= kAccEmpty && i < kDrain ? 8 : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&tmW);
    tma_prefetch_map(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), kCols);
    tmem_relinquish();
  }
  pdl_launch();
  tc_fence_before();
  if (a.parts > 1)
    cluster_sync();  // the others' shared memory may be written
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();

  if (warp == 0) {
    // ---------------- TMA producer
    const bool one = elect_one();
    uint32_t s = 0, ph = 0, issued = 0;
    bool ok = true;
    for (int tile = unit; ok && tile < a.tiles; tile += units) {
      for (int kb = k_first; kb < k_last; ++kb) {
        ok = mbar_wait(bar(kEmpty + s), ph ^ 1u, abort_flag, err, a.err_site + 1);
        if (!ok) break;
        if (one) {
          const uint32_t sw = stage0 + s * stage_bytes;
          mbar_arrive_expect_tx(bar(kFull + s), stage_bytes);
#pragma unroll
          for (int p = 0; p < kFewPanels; ++p)
            tma_load_3d(sw + p * w_panel, &tmW, bar(kFull + s), (kb * kFewPanels + p) * kBK, tile * a.height, 0);
#pragma unroll
          for (int p = 0; p < kFewPanels; ++p)
            tma_load_3d(sw + x_at + p * x_panel, &tmX, bar(kFull + s), (kb * kFewPanels + p) * kBK, 0, 0);
        }
        ++issued;
        if (++s == stages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (one && !ok) drain_ring(bar(kFull), stages, issued, issued, 0);
    __syncwarp();
  } else if (warp == 1) {
    // ---------------- MMA issuer
    const bool one = elect_one();
    uint32_t s = 0, ph = 0;
    bool ok = true;
    const uint32_t idesc = idesc_bf16_f32(128, a.x_rows, false, false);
    const uint64_t w_desc = sdesc_sw128(stage0, 16, 1024), x_desc = sdesc_sw128(stage0 + x_at, 16, 1024);
    int i = 0;
    for (int tile = unit; ok && tile < a.tiles; tile += units, ++i) {
      const int acc = i & 1;
      ok = mbar_wait(bar(kAccEmpty + acc), ((static_cast<uint32_t>(i) >> 1) & 1u) ^ 1u, abort_flag, err, a.err_site + 2);
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kFewRows);
      for (int kb = k_first; kb < k_last; ++kb) {
        ok = mbar_wait(bar(kFull + s), ph, abort_flag, err, a.err_site + 3);
        if (!ok) break;
        tc_fence_after();
        const uint64_t off = static_cast<uint64_t>(s * stage_bytes >> 4);
        if (one) {
#pragma unroll
          for (int kk = 0; kk < kFewPanels * kBK / 16; ++kk)
            umma_bf16(d, w_desc + off + (kk >> 2) * (w_panel >> 4) + (kk & 3) * 2, x_desc + off + (kk >> 2) * (x_panel >> 4) + (kk & 3) * 2,
                      idesc, static_cast<uint32_t>(kb != k_first || kk != 0));
          umma_commit(bar(kEmpty + s));
        }
        if (++s == stages) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (!ok) break;
      if (one) umma_commit(bar(kAccFull + acc));
    }
    if (one) umma_commit(bar(kDrain));
    __syncwarp();
    mbar_wait_drain(bar(kDrain), 0);
    __syncwarp();
  }
  if (a.parts == 1) {
    if (warp >= 2) {
      // ---------------- epilogue: one output column a thread, rows of X in chunks of 16 by its two warps in turn
      const int quarter = warp & 3, half = (warp - 2) >> 2, lane_row = quarter * 32 + lane;
      int i = 0;
      for (int tile = unit; tile < a.tiles; tile += units, ++i) {
        const int acc = i & 1, n = tile * a.height + lane_row;
        const bool live = lane_row < a.height && n < a.N;
        const float bias = live && a.bias ? bf16lo(a.bias[n]) : 0.0f;
        float r[16];
        auto residual = [&](int m0) {
#pragma unroll
          for (int j = 0; j < 16; ++j) r[j] = live && a.R && m0 + j < a.M ? bf16lo(a.R[(m0 + j) * a.ld_r + n]) : 0.0f;
        };
        residual(16 * half);
        const bool ok = mbar_wait(bar(kAccFull + acc), (static_cast<uint32_t>(i) >> 1) & 1u, abort_flag, err, a.err_site + 4);
        if (!__all_sync(0xFFFFFFFFu, ok)) break;
        tc_fence_after();
        const uint32_t t = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(acc * kFewRows);
#pragma unroll 1
        for (int m0 = 16 * half; m0 < a.M; m0 += 32) {
          uint32_t d[16];
          tmem_ld16(t + static_cast<uint32_t>(m0), d);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            if (m0 + j >= a.M) break;
            few_put(a, n, live, m0 + j, m0 + j + 1 < a.M ? m0 + j + 1 : -1, __uint_as_float(d[j]) + bias, __uint_as_float(d[j + 1]) + bias,
                    r[j], r[j + 1]);
          }
          if (m0 + 32 < a.M) residual(m0 + 32);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kAccEmpty + acc));
      }
    }
  } else {
    // ---------------- one tile a cluster: sums to their finishing CTAs, [part][row / parts][column]
    const int quarter = warp & 3, half = (warp - 2) >> 2, lane_row = quarter * 32 + lane, n = unit * a.height + lane_row;
    const int depth = (kFewRows + a.parts - 1) / a.parts;
    const bool live = lane_row < a.height && n < a.N;
    if (warp >= 2) {
      const bool got = mbar_wait(bar(kAccFull), 0, abort_flag, err, a.err_site + 4);
      if (__all_sync(0xFFFFFFFFu, got)) {
        tc_fence_after();
#pragma unroll 1
        for (int m0 = 16 * half; m0 < a.M; m0 += 32) {
          uint32_t d[16];
          tmem_ld16(tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(m0), d);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int m = m0 + j, to = m & (a.parts - 1);
            if (m < a.M && live)
              st_shared_cluster_f32(mapa_shared(join, static_cast<uint32_t>(to)) + static_cast<uint32_t>(((part * depth + m / a.parts) * 128 + lane_row) * 4),
                                    __uint_as_float(d[j]));
          }
        }
        tc_fence_before();
      }
    }
    __syncwarp();
    cluster_sync();  // the sums have arrived (after an abort: whatever lies there is written to Y, and the error recorded)
    if (warp >= 2 && live) {
      const float bias = a.bias ? bf16lo(a.bias[n]) : 0.0f;
#pragma unroll 1
      for (int q = 2 * half; part + q * a.parts < a.M; q += 4) {
        const int m = part + q * a.parts, m2 = m + a.parts < a.M ? m + a.parts : -1;
        const float r0 = a.R ? bf16lo(a.R[m * a.ld_r + n]) : 0.0f, r1 = a.R && m2 >= 0 ? bf16lo(a.R[m2 * a.ld_r + n]) : 0.0f;
        float z0 = 0.0f, z1 = 0.0f;
        for (int p = 0; p < a.parts; ++p) {
          const uint32_t at = join + static_cast<uint32_t>(((p * depth + q) * 128 + lane_row) * 4);
          z0 += ld_shared_f32(at);
          if (m2 >= 0) z1 += ld_shared_f32(at + 512);
        }
        few_put(a, n, true, m, m2, z0 + bias, z1 + bias, r0, r1);
      }
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, kCols);
  }
}

// ---- gZ = gY act'(Z) and the columns' sums of gZ (before its rounding).  A block owns 256 columns
// and a range of rows; lane l of each of its 8 warps owns columns 8 l .. 8 l + 7.  Bound by memory: 6 bytes an
// element.  Two rows a warp at a time and four blocks an SM: 16384 x 16384 with GeLU in 281 us (5.7 TB/s), 4096 x 8192
// with ReLU in 30.4; four rows and three blocks take 327 and 38.7, two rows and six blocks 421 and 46.
__global__ void __launch_bounds__(256, 4) lin_gz_kernel(const LinGzArgs a) {
  __shared__ float sums[8][256];
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 256 + lane * 8;
  const int64_t per = (a.M + gridDim.y - 1) / gridDim.y, r0 = per * blockIdx.y;
  const int64_t r1 = r0 + per < a.M ? r0 + per : a.M;
  const bool in = col < a.N;
  float s[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) s[e] = 0.0f;
  auto body = [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    constexpr int U = 2;
    for (int64_t r = r0 + warp; r < r1; r += 8 * U) {
      uint4 g[U], z[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool ok = r + 8 * u < r1;
        g[u] = ok ? __ldcs(reinterpret_cast<const uint4*>(a.gY + (r + 8 * u) * a.ld_gy + col)) : make_uint4(0u, 0u, 0u, 0u);
        if constexpr (ACT != ACT_NONE)
          z[u] = ok ? __ldcs(reinterpret_cast<const uint4*>(a.Z + (r + 8 * u) * a.ld_z + col)) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t gw[4] = {g[u].x, g[u].y, g[u].z, g[u].w};
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[2 * e] = bf16lo(gw[e]);
          v[2 * e + 1] = bf16hi(gw[e]);
        }
        if constexpr (ACT != ACT_NONE) {
          const uint32_t zw[4] = {z[u].x, z[u].y, z[u].z, z[u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float z0 = bf16lo(zw[e]), z1 = bf16hi(zw[e]);
            if constexpr (ACT == ACT_GELU) {
              float d0, d1;
              gelu_grad_f2(z0, z1, d0, d1);
              v[2 * e] *= d0;
              v[2 * e + 1] *= d1;
            } else {  // ReLU: a choice, so that an infinite gradient where z is cut has no effect
              v[2 * e] = z0 > 0.0f ? v[2 * e] : 0.0f;
              v[2 * e + 1] = z1 > 0.0f ? v[2 * e + 1] : 0.0f;
            }
          }
          if (r + 8 * u < r1) store8_bf16(a.gZ + (r + 8 * u) * a.ld_gz + col, v);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] += v[e];
      }
    }
  };
  if (in) {
    if (a.act == ACT_GELU)
      body(std::integral_constant<int, ACT_GELU>{});
    else if (a.act == ACT_RELU)
      body(std::integral_constant<int, ACT_RELU>{});
    else
      body(std::integral_constant<int, ACT_NONE>{});
  }
  if (!a.part) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[warp][lane * 8 + e] = s[e];
  __syncthreads();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= a.N) return;
  float t = sums[0][threadIdx.x];
#pragma unroll
  for (int k = 1; k < 8; ++k) t += sums[k][threadIdx.x];
  a.part[blockIdx.y * a.N + c] = t;
}

// The row ranges' sums in order, written or added to gbias.
__global__ void __launch_bounds__(256) lin_gbias_kernel(const float* part, int parts, int64_t n,
                                                        float* gbias, int accumulate) {
  pdl_launch();
  pdl_wait();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= n) return;
  float s = 0.0f;
#pragma unroll 8
  for (int p = 0; p < parts; ++p) s += part[p * n + c];
  gbias[c] = accumulate ? gbias[c] + s : s;
}

}  // namespace

// Estimated clocks of a product: a step of the reduction takes about 250 + 1.25 width (measured over two rounds
// of 152 tiles with 32 and 64 steps: 333 at 64 columns, 399 at 128, 488 at 192, 575 at 256; the arithmetic takes 2
// width; a CTA stages (128 + width / 2) x 128 bytes a step, 57 - 62 a clock at every width, and the shared memory that
// they are written to and read from passes 128 a clock), a round's change of tiles 8 and the last epilogue 20 a column, the start 4500, and joining cut reductions as
// below.  Where the rows of both operands begin between lines, each 128-byte row of a box is two requests to L2 and a
// step takes longer (781 at 256 columns).
LinPlan lin_plan(int64_t m, int64_t n, int64_t k) {
  constexpr int kLinQuads = 36, kLinOctets = 15;  // clusters of 4 and 8 CTAs that a GB300 keeps resident
  const int64_t m_tiles = (m + 255) / 256, kb = (k + 63) / 64;
  LinPlan best = {256, 1, 0};
  double least = 1e300;
  for (int width = 256; width >= 64; width -= 32) {
    const int64_t tiles = m_tiles * ((n + width - 1) / width);
    for (int parts = 1; parts <= 4; parts *= 2) {
      if (parts > 1 && (tiles > (parts == 2 ? kLinQuads : kLinOctets) || kb < 4 * parts)) break;
      const int64_t rounds = parts > 1 ? 1 : (tiles + kLinPairs - 1) / kLinPairs;
      const double steps = double((kb + parts - 1) / parts);
      double cost = double(rounds) * (steps * (250 + 1.25 * width) + 8.0 * width) + 20.0 * width;
      if (parts > 1) cost += (parts == 2 ? 1200.0 : 3000.0) + 45.0 * width * double(m < 256 ? m : 256) / 256;
      if (cost < least) {
        least = cost;
        best = {width, parts, static_cast<int>(parts > 1 || tiles < kLinPairs ? tiles : kLinPairs)};
      }
    }
  }
  return best;
}

cudaError_t launch_linear(int kind, const LinMaps& m, LinArgs a, cudaStream_t st) {
  if (a.units == 0) return cudaSuccess;
  const int b_rows = kind == LIN_FWD ? a.width / 2 : (a.width / 2 + 63) / 64 * 64;
  a.stage_bytes = (a.a_rows + b_rows) * 128;  // both multiples of 8 rows: swizzle atoms stay aligned
  a.stages = kLinRing / a.stage_bytes < kLinMaxStages ? kLinRing / a.stage_bytes : kLinMaxStages;
  switch (kind) {
    case LIN_FWD: return launch_linear_t<false, false>(m, a, st);
    case LIN_GX: return launch_linear_t<false, true>(m, a, st);
    case LIN_GW: return launch_linear_t<true, true>(m, a, st);
    default: return cudaErrorInvalidValue;
  }
}

// Estimated clocks: a stage (128 of the reduction) takes about 300 + 4.5 height + 2 x_rows, all of W 1765 elements a clock
// from memory, joining 700 + 55 a row sent and 150 a row finished.  Taller tiles with a cut reduction against lower ones
// without, us: one row, 4096 x 4096 7.6 (four parts) / 9.0 (two) / 11.4, 4096 x 16384 23.5 / 24.5 / 37.8, 6144 x 4096
// 11.2 (two) / 12.4; 64 rows, 6144 x 4096 16.9 (two) / 14.9, 4096 x 4096 13.5 (four) / 15.3.
void lin_few_plan(int64_t m, int64_t n, int64_t k, LinFewArgs* a) {
  constexpr int kClusters[3] = {152, 76, 36};  // clusters of 1, 2 and 4 CTAs that a GB300 keeps resident
  const int64_t kb = (k + 64 * kFewPanels - 1) / (64 * kFewPanels);
  a->k_blocks = static_cast<int32_t>(kb);
  a->x_rows = static_cast<int32_t>((m + 15) / 16 * 16);
  double least = 1e300;
  for (int i = 0; i < 3; ++i) {
    const int64_t parts = int64_t(1) << i, most = kClusters[i];
    if (parts > 1 && (n > most * 128 || kb < 4 * parts)) break;
    const int64_t rounds = (n + most * 128 - 1) / (most * 128), share = (n + most * rounds - 1) / (most * rounds);
    const int64_t height = (share + 7) / 8 * 8, tiles = (n + height - 1) / height;
    const double steps = double(rounds * ((kb + parts - 1) / parts)), dram = double(n) * double(k) / 1765.0;
    double cost = steps * (300 + 4.5 * double(height) + 2.0 * double(a->x_rows));
    if (cost < dram) cost = dram;
    if (parts > 1) cost += 700.0 + double(m) * (55.0 + 150.0 / double(parts));
    if (cost < least) {
      least = cost;
      a->height = static_cast<int32_t>(height);
      a->parts = static_cast<int32_t>(parts);
      a->tiles = static_cast<int32_t>(tiles);
      a->units = static_cast<int32_t>(tiles < most ? tiles : most);
    }
  }
}

cudaError_t launch_linear_few(const CUtensorMap& w, const CUtensorMap& x, LinFewArgs a, cudaStream_t st) {
  if (a.units == 0) return cudaSuccess;
  static std::atomic<bool> ready_of[kMaxDevices];  // the shared-memory opt-in, per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!ready_of[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(linear_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem);
    if (e != cudaSuccess) return e;
    ready_of[dev].store(true, std::memory_order_release);
  }
  a.stage_bytes = kFewPanels * (a.height + a.x_rows) * 128;  // both multiples of 8 rows: swizzle atoms stay aligned
  a.stages = kFewRing / a.stage_bytes < kFewStages ? kFewRing / a.stage_bytes : kFewStages;
  return launch_pdl(linear_few_kernel, dim3(static_cast<unsigned>(a.parts * a.units)), dim3(kLinThreads), kFewSmem, a.parts, st, w, x, a);
}

int lin_gz_row_blocks(int64_t m, int64_t n) {
  // about eight blocks of 256 threads an SM, and 64 rows a block where there are that many
  const int64_t cols = (n + 255) / 256, want = (int64_t(152) * 8 + cols - 1) / cols, most = (m + 63) / 64;
  return static_cast<int>(want < most ? want : most);
}

cudaError_t launch_lin_gz(const LinGzArgs& a, cudaStream_t st) {
  const int rb = lin_gz_row_blocks(a.M, a.N);
  if (rb == 0 || a.N == 0) return cudaSuccess;
  return launch_pdl(lin_gz_kernel, dim3(static_cast<unsigned>((a.N + 255) / 256), static_cast<unsigned>(rb)), dim3(256), 0, 1, st, a);
}

cudaError_t launch_lin_gbias(const float* part, int64_t m, int64_t n, float* gbias, int accumulate, cudaStream_t st) {
  return launch_pdl(lin_gbias_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, 1, st, part,
                    lin_gz_row_blocks(m, n), n, gbias, accumulate);
}

cudaError_t take_linear_error(int* code) { return take_error_word(code); }

}  // namespace dm
