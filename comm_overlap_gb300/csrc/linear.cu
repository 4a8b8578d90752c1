// linear.cu -- the linear layer's products: D = A . B^T (bf16 operands, either one contiguous along
// the reduction or along its rows, fp32 accumulation) with an epilogue that adds a bias, keeps the
// pre-activation, applies an activation, adds a residual and rounds once to bf16; and the column
// pass of the backward (gZ = gY act'(Z), bias gradient).
//
// The product runs on CTA pairs (cluster of 2, tcgen05.mma.cta_group::2, 256 x 256 tiles, 64 elements
// of the reduction a step through a 6-stage TMA ring), one pair per two SMs:
//   warp 0 (one lane)  TMA producer of this CTA's 128 rows of A and its 128 rows of B
//   warp 1 (one lane of the leader)  MMA issuer, two 256-column accumulators in TMEM
//   warps 2-9          epilogue, two per TMEM lane quarter with 128 columns each, one row a thread
// Work split: while whole rounds of tiles (one per pair) remain, a pair takes tiles unit, unit + units,
// ...  The last round's `rest` tiles, if they would leave pairs idle, are laid end to end along the
// reduction and cut into equal shares of `q` steps, one per pair; a share covers the end of one tile
// and perhaps the beginning of the next.  The pair that computes a tile's end adds the other shares'
// fp32 partials (in memory, one slot a pair) in their order along the reduction and runs the
// epilogue, so results do not depend on timing.  A pair publishes its partial before it does
// anything else and waits, last of all, only for pairs of lower index, which were launched before
// it: no two pairs wait for each other, whatever else occupies the GPU.
#include "gemm.cuh"
#include "ops.h"

namespace dm {

namespace {

constexpr int kLinThreads = 320;
constexpr int kLinStages = 6;
constexpr int kLinStageBytes = 32768;  // 128 x 64 bf16 of A, then of B
constexpr int kLinWarpBytes = 4096;    // an epilogue warp's boxes: Y, Z (32 x 32 bf16 each)
constexpr int kLinSmem = 1024 + kCtrlBytes + kLinStages * kLinStageBytes + 8 * kLinWarpBytes;
static_assert(kLinSmem <= 232448, "shared memory beyond the per-CTA limit");

// A pair's share of the last round: [k0, k1) of one tile.
struct LinSeg {
  int tile, k0, k1;
};

struct LinWork {
  int units, unit, full, kb;
  LinSeg pub, fin;  // the part published for another pair (k1 > k0), the part finished here
  int helpers;      // pairs unit - helpers .. unit - 1 hold the partials of fin's tile

  __device__ LinWork(const LinArgs& a, int unit_, int units_) : units(units_), unit(unit_), kb(a.k_blocks) {
    const int tiles = a.m_tiles * a.n_tiles;
    full = tiles / a.round;
    const int rest = tiles - full * a.round;
    const int total = rest * kb, i0 = unit * a.share, i1 = min(i0 + a.share, total);
    pub = fin = LinSeg{0, 0, 0};
    helpers = 0;
    if (i0 >= i1) return;
    const int t = i0 / kb, lo = i0 - t * kb, end = (t + 1) * kb;
    const LinSeg first{full * a.round + t, lo, min(i1, end) - t * kb};
    if (first.k1 < kb) {
      pub = first;
    } else {
      fin = first;
      helpers = unit - t * kb / a.share;
      if (i1 > end) pub = LinSeg{first.tile + 1, 0, i1 - end};
    }
  }
  // segments in the order every role walks them: the published part, whole tiles, the finished part
  __device__ int count() const { return (pub.k1 > 0 ? 1 : 0) + full + (fin.k1 > 0 ? 1 : 0); }
  __device__ LinSeg at(int i, bool& publish) const {
    publish = false;
    if (pub.k1 > 0) {
      if (i == 0) {
        publish = true;
        return pub;
      }
      --i;
    }
    if (i < full) return LinSeg{unit + i * units, 0, kb};
    return fin;
  }
};

// Tiles in groups of 8 rows of tiles, so that the operands of concurrent tiles stay in L2.
__device__ __forceinline__ void lin_tile(const LinArgs& a, int tile, int& mt, int& nt) {
  const int span = kGroupM * a.n_tiles;
  const int grp = tile / span, first = grp * kGroupM, size = min(a.m_tiles - first, kGroupM), in = tile - grp * span;
  mt = first + in % size;
  nt = in / size;
}

// Waits until the warp of the same place in pair u has written its block of u's partial slot.
__device__ __forceinline__ bool wait_flag(const uint32_t* flag, volatile int* abort_flag, int* err, int site,
                                          int lane) {
  bool ok = true;
  if (lane == 0) {
    uint64_t t0 = 0;
    for (uint32_t it = 0; ld_acquire_u32(flag) == 0; ++it) {
      if ((it & 63u) == 63u) {
        const uint64_t now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (*abort_flag || now - t0 > kWaitTimeoutNs) {
          if (!*abort_flag) atomicCAS(err, 0, site);
          *abort_flag = 1;
          ok = false;
          break;
        }
      }
    }
  }
  ok = __shfl_sync(0xFFFFFFFFu, ok ? 1 : 0, 0) != 0;
  if (ok) (void)ld_acquire_u32(flag);
  return ok;
}

template <bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                  const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmZ, const LinArgs a) {
  constexpr int S = kLinStages;
  constexpr uint32_t kIdesc = idesc_bf16_f32(256, 256, A_MN, B_MN);
  constexpr int kFull = 0, kEmpty = S, kAccFull = 2 * S, kAccEmpty = 2 * S + 2, kDrain = 2 * S + 4,
                kPeerCount = 2 * S + 5;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + 512);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + 516);
  volatile uint32_t* peer_issued = reinterpret_cast<volatile uint32_t*>(smem + 520);
  const uint32_t bar0 = smem_u32(smem), stage0 = smem_u32(smem + kCtrlBytes);
  auto bar = [bar0](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int unit = static_cast<int>(blockIdx.x >> 1), units = static_cast<int>(gridDim.x >> 1);
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
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const LinWork w(a, unit, units);
  const int nseg = w.count();

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer
      uint32_t s = 0, ph = 0, issued = 0;
      bool ok = true, pub;
      for (int i = 0; ok && i < nseg; ++i) {
        const LinSeg g = w.at(i, pub);
        int mt, nt;
        lin_tile(a, g.tile, mt, nt);
        const int m0 = mt * 256 + static_cast<int>(rank) * 128, n0 = nt * 256 + static_cast<int>(rank) * 128;
        for (int kb = g.k0; kb < g.k1; ++kb) {
          if (!mbar_wait(bar(kEmpty + s), ph ^ 1u, abort_flag, err, a.err_site + 1)) {
            ok = false;
            break;
          }
          const uint32_t sa = stage0 + s * kLinStageBytes, sb = sa + kLinStageBytes / 2;
          const uint32_t fb = mapa_shared(bar(kFull + s), 0);  // the leader's barrier counts both CTAs' bytes
          const int k0 = kb * kBK;
          if (leader) mbar_arrive_expect_tx(bar(kFull + s), 2u * kLinStageBytes);
          if constexpr (!A_MN) {
            tma_load_3d_pair(sa, &tmA, fb, k0, m0, 0);
          } else {
            tma_load_3d_pair(sa, &tmA, fb, m0, k0, 0);
            tma_load_3d_pair(sa + 8192, &tmA, fb, m0 + 64, k0, 0);
          }
          if constexpr (!B_MN) {
            tma_load_3d_pair(sb, &tmB, fb, k0, n0, 0);
          } else {
            tma_load_3d_pair(sb, &tmB, fb, n0, k0, 0);
            tma_load_3d_pair(sb + 8192, &tmB, fb, n0 + 64, k0, 0);
          }
          ++issued;
          if (++s == S) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      // both CTAs' copies have landed before the pair leaves, also after an abort (gemm.cuh)
      if (!leader) {
        st_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t*>(peer_issued)), 0), issued);
        mbar_arrive_cluster(mapa_shared(bar(kPeerCount), 0));
      } else if (mbar_wait_cluster_acquire(bar(kPeerCount), 0, kPeerCountTimeoutNs)) {
        const uint32_t peer = *peer_issued;
        if (!ok || peer != issued || *abort_flag) drain_pair_ring<S>(bar(kFull), issued, peer, kLinStageBytes);
      } else {
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < kPeerCopyGraceNs) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---------------- MMA issuer for both CTAs
      uint32_t s = 0, ph = 0;
      bool ok = true, pub;
      for (int i = 0; ok && i < nseg; ++i) {
        const LinSeg g = w.at(i, pub);
        const int acc = i & 1;
        if (!mbar_wait(bar(kAccEmpty + acc), ((static_cast<uint32_t>(i) >> 1) & 1u) ^ 1u, abort_flag, err,
                       a.err_site + 2))
          break;
        tc_fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kBN);
        for (int kb = g.k0; kb < g.k1; ++kb) {
          if (!mbar_wait(bar(kFull + s), ph, abort_flag, err, a.err_site + 3)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = stage0 + s * kLinStageBytes, sb = sa + kLinStageBytes / 2;
#pragma unroll
          for (int kk = 0; kk < kBK / 16; ++kk) {
            const uint64_t ad = A_MN ? sdesc_sw128(sa + kk * 2048, 8192, 1024) : sdesc_sw128(sa + kk * 32, 16, 1024);
            const uint64_t bd = B_MN ? sdesc_sw128(sb + kk * 2048, 8192, 1024) : sdesc_sw128(sb + kk * 32, 16, 1024);
            umma_bf16_pair(d, ad, bd, kIdesc, static_cast<uint32_t>(kb != g.k0 || kk != 0));
          }
          umma_commit_pair_multicast(bar(kEmpty + s), 0x3);
          if (++s == S) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair_multicast(bar(kAccFull + acc), 0x3);
      }
      umma_commit_pair(bar(kDrain));
      mbar_wait_drain(bar(kDrain), 0);
    }
  } else {
    // ---------------- epilogue: rows of the warp's TMEM lane quarter, 128 of the tile's columns
    const int ew = warp - 2, quarter = warp & 3, half = ew >> 2;
    const uint32_t box_y = stage0 + S * kLinStageBytes + static_cast<uint32_t>(ew) * kLinWarpBytes, box_z = box_y + 2048u;
    const uint32_t rsw = static_cast<uint32_t>(lane) * 64u, rx = (static_cast<uint32_t>(lane) >> 1) & 3u;
    const uint32_t tq = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(half * 128);
    // this warp's block in a partial slot: 32 pieces of 16 bytes a lane, 512 bytes a piece
    const int64_t wofs = static_cast<int64_t>(rank * 8 + static_cast<uint32_t>(ew)) * kSlotWarpBytes + lane * 16;
    const uint32_t wflag = rank * 8 + static_cast<uint32_t>(ew);
    auto slot = [&](int u) { return a.part + static_cast<int64_t>(u) * kSlotBytes + wofs; };
    bool stored = false, pub, ok = true;
    for (int i = 0; ok && i < nseg; ++i) {
      const LinSeg g = w.at(i, pub);
      int mt, nt;
      lin_tile(a, g.tile, mt, nt);
      const int row0 = mt * 256 + static_cast<int>(rank) * 128 + quarter * 32, row = row0 + lane;
      const int colw = nt * 256 + half * 128;
      const int acc = i & 1;
      ok = mbar_wait(bar(kAccFull + acc), (static_cast<uint32_t>(i) >> 1) & 1u, abort_flag, err, a.err_site + 4);
      if (!__all_sync(0xFFFFFFFFu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t tacc = tq + static_cast<uint32_t>(acc * kBN);
      const bool live = row0 < a.M && colw < a.N;  // something of this warp's part is inside D
      const int nhelp = (!pub && i == nseg - 1 && w.fin.k1 > 0) ? w.helpers : 0;
      for (int u = unit - nhelp; ok && live && u < unit; ++u)
        ok = wait_flag(a.flags + u * 16 + wflag, abort_flag, err, a.err_site + 6, lane);
      if (!ok) break;
#pragma unroll 1
      for (int cc = 0; cc < 128; cc += 32) {
        const int col = colw + cc;
        if (!live || col >= a.N) break;
        uint32_t r[32];
        tmem_ld32(tacc + static_cast<uint32_t>(cc), r);
        if (pub) {
          tmem_ld_wait();
          if (row < a.M) {
            uint4* p = reinterpret_cast<uint4*>(slot(unit)) + cc / 4 * 32;
#pragma unroll
            for (int q = 0; q < 8; ++q)
              __stcg(p + q * 32, make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]));
          }
          continue;
        }
        uint4 bias[4], res[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const bool in = col + 8 * q < a.N;
          bias[q] = in && a.bias ? *reinterpret_cast<const uint4*>(a.bias + col + 8 * q) : make_uint4(0u, 0u, 0u, 0u);
          res[q] = in && a.R && row < a.M
                       ? *reinterpret_cast<const uint4*>(a.R + static_cast<int64_t>(row) * a.ld_r + col + 8 * q)
                       : make_uint4(0u, 0u, 0u, 0u);
        }
        tmem_ld_wait();
        for (int u = unit - nhelp; u < unit; ++u) {
          if (row >= a.M) break;
          const uint4* p = reinterpret_cast<const uint4*>(slot(u)) + cc / 4 * 32;
          uint4 v[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) v[q] = __ldcg(p + q * 32);
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            r[4 * q] = __float_as_uint(__uint_as_float(r[4 * q]) + __uint_as_float(v[q].x));
            r[4 * q + 1] = __float_as_uint(__uint_as_float(r[4 * q + 1]) + __uint_as_float(v[q].y));
            r[4 * q + 2] = __float_as_uint(__uint_as_float(r[4 * q + 2]) + __uint_as_float(v[q].z));
            r[4 * q + 3] = __float_as_uint(__uint_as_float(r[4 * q + 3]) + __uint_as_float(v[q].w));
          }
        }
        // Z = D + bias; Y = act(Z) + R, each rounded once from fp32
        uint32_t yz[2][16];
        auto finish = [&](auto act) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const uint32_t bw[4] = {bias[q].x, bias[q].y, bias[q].z, bias[q].w};
            const uint32_t rw[4] = {res[q].x, res[q].y, res[q].z, res[q].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float z0 = __uint_as_float(r[8 * q + 2 * e]) + bf16lo(bw[e]);
              const float z1 = __uint_as_float(r[8 * q + 2 * e + 1]) + bf16hi(bw[e]);
              yz[1][4 * q + e] = pack_bf16x2(z0, z1);
              yz[0][4 * q + e] = pack_bf16x2(act_fwd(decltype(act)::value, z0) + bf16lo(rw[e]),
                                             act_fwd(decltype(act)::value, z1) + bf16hi(rw[e]));
            }
          }
        };
        if (a.act == ACT_GELU)
          finish(std::integral_constant<int, ACT_GELU>{});
        else if (a.act == ACT_RELU)
          finish(std::integral_constant<int, ACT_RELU>{});
        else
          finish(std::integral_constant<int, ACT_NONE>{});
        if (lane == 0 && stored) bulk_wait_group_read<0>();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t off = rsw + ((static_cast<uint32_t>(j) ^ rx) << 4);
          st_shared_v4(box_y + off, yz[0][4 * j], yz[0][4 * j + 1], yz[0][4 * j + 2], yz[0][4 * j + 3]);
          if (a.save) st_shared_v4(box_z + off, yz[1][4 * j], yz[1][4 * j + 1], yz[1][4 * j + 2], yz[1][4 * j + 3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_3d(&tmY, box_y, col, row0, 0);
          if (a.save) tma_store_3d(&tmZ, box_z, col, row0, 0);
          bulk_commit_group();
        }
        stored = true;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (pub) {
          __threadfence();
          asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(a.flags + unit * 16 + wflag), "r"(1u) : "memory");
        }
        mbar_arrive_cluster_relaxed(mapa_shared(bar(kAccEmpty + acc), 0));
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

// Steps of the reduction below which a share of the last round is not cut further.
constexpr int kMinShare = 8;

// How a product of `tiles` tiles of `kb` steps is laid over at most `pairs` pairs.
struct LinSplit {
  int units, round, share;
  bool split;
};
LinSplit lin_split(int64_t tiles, int kb, int pairs) {
  LinSplit s;
  s.round = pairs;
  const int64_t full = tiles / pairs, rest = tiles - full * pairs;
  int64_t q = (rest * kb + pairs - 1) / pairs;
  if (q < kMinShare) q = kMinShare;
  if (rest == 0 || q * 8 > int64_t(kb) * 7) q = kb;  // little to gain: whole tiles
  s.share = static_cast<int>(q);
  const int64_t parts = (rest * kb + q - 1) / q;
  s.units = static_cast<int>(full > 0 ? pairs : parts);
  s.split = rest > 0 && q < kb;
  return s;
}

template <bool A_MN, bool B_MN>
cudaError_t launch_linear_t(const LinMaps& m, LinArgs a, cudaStream_t st) {
  auto fn = linear_kernel<A_MN, B_MN>;
  static std::atomic<int> pairs_of[kMaxDevices];  // co-resident pairs per device; 0 = not set up
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kLinThreads);
  cfg.dynamicSmemBytes = kLinSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int pairs = pairs_of[dev].load(std::memory_order_acquire);
  if (pairs == 0) {
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kLinSmem);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(2);
    e = cudaOccupancyMaxActiveClusters(&pairs, fn, &cfg);
    if (e != cudaSuccess) return e;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    if (pairs > kLinPairs) pairs = kLinPairs;  // what the workspace is sized for
    pairs_of[dev].store(pairs, std::memory_order_release);
  }
  const LinSplit s = lin_split(int64_t(a.m_tiles) * a.n_tiles, a.k_blocks, pairs);
  if (s.units == 0) return cudaSuccess;
  a.round = s.round;
  a.share = s.share;
  if (s.split) {
    e = cudaMemsetAsync(a.flags, 0, kLinPairs * 64, st);
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3(2 * s.units);
  return cudaLaunchKernelEx(&cfg, fn, m.a, m.b, m.y, m.z, a);
}

// ---- gZ = gY act'(Z) and the columns' sums of gZ (before its rounding).  A block owns 256 columns
// and a range of rows; lane l of each of its 8 warps owns columns 8 l .. 8 l + 7.
__global__ void __launch_bounds__(256) lin_gz_kernel(const LinGzArgs a) {
  __shared__ float sums[8][256];
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
    constexpr int U = 4;
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
            v[2 * e] *= act_grad(ACT, bf16lo(zw[e]));
            v[2 * e + 1] *= act_grad(ACT, bf16hi(zw[e]));
          }
          if (r + 8 * u < r1) store8_bf16(a.gZ + (r + 8 * u) * a.N + col, v);
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
__global__ void __launch_bounds__(256) lin_gbias_kernel(const float* __restrict__ part, int parts, int64_t n,
                                                        float* gbias, int accumulate) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= n) return;
  float s = 0.0f;
#pragma unroll 8
  for (int p = 0; p < parts; ++p) s += part[p * n + c];
  gbias[c] = accumulate ? gbias[c] + s : s;
}

}  // namespace

int64_t lin_scratch_bytes(int64_t m, int64_t n, int64_t k) {
  const int64_t tiles = ((m + 255) / 256) * ((n + 255) / 256);
  // a device may keep fewer pairs resident than kLinPairs: any last round may then be split
  return tiles == 0 || k <= kMinShare * kBK ? 0 : int64_t(kLinPairs) * (kSlotBytes + 64);
}

cudaError_t launch_linear(int kind, const LinMaps& m, LinArgs a, void* scratch, cudaStream_t st) {
  a.part = static_cast<uint8_t*>(scratch);
  a.flags = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(scratch) + int64_t(kLinPairs) * kSlotBytes);
  switch (kind) {
    case LIN_FWD: return launch_linear_t<false, false>(m, a, st);
    case LIN_GX: return launch_linear_t<false, true>(m, a, st);
    case LIN_GW: return launch_linear_t<true, true>(m, a, st);
    default: return cudaErrorInvalidValue;
  }
}

int lin_gz_row_blocks(int64_t m, int64_t n) {
  // about eight blocks of 256 threads an SM, and 64 rows a block where there are that many
  const int64_t cols = (n + 255) / 256, want = (int64_t(152) * 8 + cols - 1) / cols, most = (m + 63) / 64;
  return static_cast<int>(want < most ? want : most);
}

cudaError_t launch_lin_gz(const LinGzArgs& a, cudaStream_t st) {
  const int rb = lin_gz_row_blocks(a.M, a.N);
  if (rb == 0 || a.N == 0) return cudaSuccess;
  lin_gz_kernel<<<dim3(static_cast<unsigned>((a.N + 255) / 256), static_cast<unsigned>(rb)), 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_lin_gbias(const float* part, int64_t m, int64_t n, float* gbias, int accumulate, cudaStream_t st) {
  lin_gbias_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, st>>>(part, lin_gz_row_blocks(m, n), n, gbias,
                                                                            accumulate);
  return cudaGetLastError();
}

cudaError_t take_linear_error(int* code) { return take_error_word(code); }

}  // namespace dm
