// Products grouped by expert on sm_103a tensor cores: rows sorted by group, each
// group with its own matrix (forward and input gradient), or each group with its
// own result over the group's rows (weights' gradient).  The groups' bounds are
// on the device only.
//
// A cluster of two CTAs computes units of 256 columns x up to 256 rows of C with
// tcgen05.mma.cta_group::2.kind::f16.  The columns of C are the MMA's M side,
// the rows its N side, which goes in steps of 32: a group's last, ragged unit
// costs MMAs and loads for its rows only, where 256 rows on the M side would be
// padded in full.  A TMEM lane is a column of C, so that a warp stores 32
// consecutive columns of a row, whatever C's alignment, and the rows of the next
// group are simply not stored.
//
// Roles (384 threads): warp 0 loads both operands by TMA, warp 1 issues the MMAs
// (even CTA), warp 2 clears the rows past a group's end (weights' gradient),
// warps 4-11 drain the accumulators and store.
//
// Few units would leave most SMs idle: up to four pairs of a cluster then share a unit's K
// and add their sums through distributed shared memory, in their order.
//
// Measured (8 experts of 4096 x 4096, 8192 rows, in a graph of twelve): forward 162 us (1.70
// PFLOP/s; back to back for longer, under the power limit, 184); weights' gradient in FP32
// 206, in BF16 171.  What bounds them is what moves
// between L2 and the SMs, 128 KB for each k-tile of a unit and the results: forward without
// loads 134 us, the gradients without stores 148 and 138, with one MMA of eight 180 and 142.
// Small groups read each weight once: 64 rows of 32 experts, 2048 x 2048, 35 us (6.2 TB/s).
//
// FP32 sums.  The MMA truncates the running sum at every 16-deep step, so a unit
// is summed in segments (GroupParams::seg), which the draining warps add in
// registers, rounding to nearest; the two accumulators in tensor memory let that
// overlap the next segment.
#include "group_sched.cuh"

namespace dgemm {
namespace {

constexpr int BK = kGroupBK;
constexpr int kThreads = 384;
constexpr int kEpiWarp = 4, kEpiWarps = kGroupEpiWarps;

// A stage: the CTA's 128 columns of C and its half of a tile's rows, BK deep.  K-major
// operands are two blocks of 64 k (128-byte swizzled rows), MN-major ones two blocks 64
// wide with a row for each k.  kRows: most rows of a tile, 256, or 64 where groups are
// small: its stages take less room, so that there are more of them, and five stages of
// weights in flight rather than three make 64 rows of 32 experts, 2048 x 2048, 40.3 ->
// 38.1 us (256 rows 53.2 -> 49.2, 2048 56.2 -> 51.9).
constexpr uint32_t kBlock = 128 * 128;
constexpr uint32_t kSide = 2 * kBlock;
constexpr uint32_t kTmemCols = 512;                       // two accumulators
constexpr uint32_t kTableBytes = (sizeof(GroupTables) + 15) / 16 * 16;
template <int kRows>
struct Layout {
  static constexpr uint32_t kNBlock = kRows / 2 * 128;
  static constexpr uint32_t kStage = kSide + 2 * kNBlock;
  static constexpr int S = kRows == 256 ? 3 : 5;
  static constexpr uint32_t kSmem = S * kStage + kTableBytes + 512 + 1024;
  static_assert(kSmem <= 232448, "shared memory");
};

template <int S>
struct alignas(8) Barriers {
  uint64_t full[S];       // even CTA: both CTAs' operands are there
  uint64_t empty[S];      // the MMAs on stage s are done
  uint64_t tail[S];       // weights: this CTA's part of a stage that ends its group
  uint64_t acc_full[2];
  uint64_t acc_empty[2];  // even CTA
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* desc,
                                                 uint32_t cluster_bar, int32_t x, int32_t y,
                                                 int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(desc)), "r"(cluster_bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

template <typename T, typename TC, int kKind, int kRows>
__global__ void __launch_bounds__(kThreads, 1)
    group_kernel(const __grid_constant__ CUtensorMap tmM, const __grid_constant__ CUtensorMap tmN,
                 const __grid_constant__ CUtensorMap tmN16, const GroupParams p) {
  using L = Layout<kRows>;
  constexpr int S = L::S;
  constexpr uint32_t kStage = L::kStage;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* const base = align_smem_1024(smem_raw);
  GroupTables& tables = *reinterpret_cast<GroupTables*>(base + S * kStage);
  auto* bars = reinterpret_cast<Barriers<S>*>(base + S * kStage + kTableBytes);
  static_assert(sizeof(Barriers<S>) <= 512, "barrier block must fit its reserved space");
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // A cluster is a pair, or up to four, which share a unit's K.
  const uint32_t crank = cluster_ctarank();
  const uint32_t rank = crank & 1u;          // 0: issues the pair's MMAs
  const uint32_t leader = crank & ~1u;
  const uint16_t both = (uint16_t)(0x3u << leader);
  const int parts = 1 << p.log_parts, part = (int)(crank >> 1);
  const int clusters = (int)gridDim.x >> (1 + p.log_parts);
  const int cluster = (int)blockIdx.x >> (1 + p.log_parts);
  constexpr bool kWeights = kKind == kGroupWeights;
  constexpr bool kMK = kKind == kGroupForward;   // the M side is K-major
  constexpr uint32_t kAb = __is_same(T, __half) ? 0u : 1u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&bars->full[s]), kWeights ? 2 : 1);
      mbar_init(smem_u32(&bars->empty[s]), 1);
      mbar_init(smem_u32(&bars->tail[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&bars->acc_full[b]), 1);
      mbar_init(smem_u32(&bars->acc_empty[b]), 2 * kEpiWarps);
    }
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmM);
    tma_prefetch_desc(&tmN);
    if constexpr (!kWeights) tma_prefetch_desc(&tmN16);
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(&bars->tmem_base), kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();     // the peer's barriers are initialised
  tc_fence_after();
  wait_prior_grids();
  allow_dependent_grids();
  if (warp == 2) group_tables<kKind, kRows>(p, tables);
  __syncthreads();
  const uint32_t tmem_base = bars->tmem_base;
  const int units = tables.units;

  uint32_t issued = 0;
  if (warp == 0) {
    if (elect_one()) {
      // ---------------------------------------------- loads (both CTAs)
      RingPos<S> pos;
      uint32_t it = 0;
      bool ok = true;
      for (int u = cluster; u < units && ok; u += clusters) {
        const GroupUnit w = group_unit<kKind, kRows>(u, p, tables);
        const int half = w.mma_rows / 2;                 // rows of C that this CTA loads
        const int row = w.row + (int)rank * half;
        const int col = w.col + (int)rank * 128;
        const int z = w.g * p.zmul;
        const int k_first = group_part_first(w.nk, part, p);
        const int k_last = group_part_first(w.nk, part + 1, p);
        for (int kt = k_first; kt < k_last; ++kt, ++it, pos.next()) {
          const uint32_t s = pos.slot;
          ok = role_wait(smem_u32(&bars->empty[s]), pos.parity ^ 1u, p.fault, p.timeout_ns,
                         &bars->abort, kFaultTcProducerWait, true);
          if (!ok) break;
          const uint32_t sm = smem_u32(base + s * kStage), sn = sm + kSide;
          const uint32_t full = smem_u32(&bars->full[s]);
          const uint32_t fb = mapa_shared(full, leader);
          if constexpr (kWeights) {
            const int k = w.k0 + kt * BK;
            const int valid = w.k_end - k;               // rows of the group from k on
            const int deep = valid > 64 ? 2 : 1, wide = half > 64 ? 2 : 1;
            const uint32_t bytes = (uint32_t)(deep * (2 + wide)) * (kBlock / 2);
            const bool ragged = valid < BK && (valid & 15) != 0;
            const uint32_t tail = smem_u32(&bars->tail[s]);
            if (ragged)
              mbar_arrive_expect_tx(tail, bytes);
            else if (rank == 0)
              mbar_arrive_expect_tx(full, 2 * bytes);
            else
              mbar_arrive_any_cta(fb);
            for (int d = 0; d < deep; ++d) {
              for (int j = 0; j < 2; ++j) {
                const uint32_t to = sm + j * kBlock + d * (kBlock / 2);
                if (ragged)
                  tma_load_2d(to, &tmM, tail, col + j * 64, k + d * 64);
                else
                  tma_load_2d_pair(to, &tmM, fb, col + j * 64, k + d * 64);
              }
              for (int j = 0; j < wide; ++j) {
                const uint32_t to = sn + j * kBlock + d * (kBlock / 2);
                if (ragged)
                  tma_load_2d(to, &tmN, tail, row + j * 64, k + d * 64);
                else
                  tma_load_2d_pair(to, &tmN, fb, row + j * 64, k + d * 64);
              }
            }
          } else {
            if (rank == 0)
              mbar_arrive_expect_tx(full, 2 * (kSide + (uint32_t)half * 256));
            const int k = kt * BK;
            for (int j = 0; j < 2; ++j) {
              if constexpr (kMK)
                tma_load_3d_pair(sm + j * kBlock, &tmM, fb, k + j * 64, col, z);
              else
                tma_load_3d_pair(sm + j * kBlock, &tmM, fb, col + j * 64, k, z);
            }
            for (int j = 0; j < 2; ++j) {
              if (half == kRows / 2) {
                tma_load_2d_pair(sn + j * L::kNBlock, &tmN, fb, k + j * 64, row);
              } else {
                for (int r = 0; r < half; r += 16)
                  tma_load_2d_pair(sn + j * L::kNBlock + r * 128, &tmN16, fb, k + j * 64, row + r);
              }
            }
          }
          issued = it + 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      // ---------------------------------------------- MMA issuer (even CTA)
      RingPos<S> pos;
      bool ready = false;
      uint32_t seg = 0;
      bool ok = true;
      for (int u = cluster; u < units && ok; u += clusters) {
        const GroupUnit w = group_unit<kKind, kRows>(u, p, tables);
        const uint32_t idesc = instr_desc(kAb, 256, (uint32_t)w.mma_rows, kMK ? 0u : 1u,
                                          kWeights ? 1u : 0u);
        const int k_first = group_part_first(w.nk, part, p);
        const int k_last = group_part_first(w.nk, part + 1, p);
        for (int k0 = k_first; k0 < k_last && ok; k0 += p.seg, ++seg) {
          const int k1 = min(k0 + p.seg, k_last);
          const uint32_t b = seg & 1;
          ok = role_wait(smem_u32(&bars->acc_empty[b]), ((seg >> 1) & 1u) ^ 1u, p.fault,
                         p.timeout_ns, &bars->abort, kFaultTcMmaWait, true);
          if (!ok) break;
          tc_fence_after();
          for (int kt = k0; kt < k1; ++kt) {
            const uint32_t st = smem_u32(base + pos.slot * kStage);
            const uint32_t freed = smem_u32(&bars->empty[pos.slot]);
            ok = ready || role_wait(smem_u32(&bars->full[pos.slot]), pos.parity, p.fault,
                                    p.timeout_ns, &bars->abort, kFaultTcMmaWait, true);
            if (!ok) break;
            tc_fence_after();
            pos.next();
            ready = mbar_try_wait(smem_u32(&bars->full[pos.slot]), pos.parity);
            // MN-major blocks step by 16 rows of 128 bytes per 16 of K, K-major
            // ones by 32 bytes, 64 to a block.
            const uint32_t mlo = desc_lo(st, kMK ? 16 : kBlock);
            const uint32_t nlo = desc_lo(st + kSide, kWeights ? kBlock : 16);
            // (Whole steps past the group's end are left out, not only cleared:
            // nothing has loaded them.)
            const int steps = kWeights ? min((w.k_end - w.k0 - kt * BK + 15) / 16, BK / 16)
                                       : BK / 16;
#pragma unroll
            for (int k = 0; k < BK / 16; ++k)
              if (!kWeights || k < steps)
                mma_f16_pair_lo(
                    tmem_base + b * 256,
                    mlo + ((kMK ? (k >> 2) * kBlock + (k & 3) * 32 : k * 2048) >> 4),
                    nlo + ((kWeights ? k * 2048 : (k >> 2) * L::kNBlock + (k & 3) * 32) >> 4), idesc,
                    (kt > k0 || k > 0) ? 1u : 0u);
            mma_commit_pair_multicast(freed, both);
          }
          if (!ok) break;
          mma_commit_pair_multicast(smem_u32(&bars->acc_full[b]), both);
        }
      }
      // The other CTA's last arrivals have come before this one may leave.
      for (uint32_t i = seg > 2 ? seg - 2 : 0; ok && i < seg; ++i)
        ok = role_wait(smem_u32(&bars->acc_empty[i & 1]), (i >> 1) & 1u, p.fault, p.timeout_ns,
                       &bars->abort, kFaultTcMmaWait, true);
    }
    __syncwarp();
  } else if (warp == 2) {
    if constexpr (kWeights) {
      // ------------------------------------------------ ragged ends (both CTAs)
      // The rows of the next group in a group's last 16 are cleared in both
      // operands (zero times a NaN is not zero).
      uint32_t it = 0, uses = 0;   // a bit per slot: the parity of its next use
      bool ok = true;
      for (int u = cluster; u < units && ok; u += clusters) {
        const GroupUnit w = group_unit<kKind, kRows>(u, p, tables);
        const int k_first = group_part_first(w.nk, part, p);
        const int k_last = group_part_first(w.nk, part + 1, p);
        it += (uint32_t)(k_last - k_first);
        const int valid = w.k_end - w.k0 - (w.nk - 1) * BK;
        if (k_last == k_first || k_last != w.nk || (valid & 15) == 0) continue;
        const uint32_t s = (it - 1) % S;
        ok = role_wait_lanes(smem_u32(&bars->tail[s]), (uses >> s) & 1u, p.fault, p.timeout_ns,
                             &bars->abort, kFaultTcProducerWait);
        if (!ok) break;
        uses ^= 1u << s;
        const int blocks = w.mma_rows / 2 > 64 ? 4 : 3;
        const int clear = 16 - (valid & 15);
        for (int i = lane; i < blocks * clear * 8; i += 32) {
          const int row = valid + (i >> 3) % clear, b = (i >> 3) / clear;
          *reinterpret_cast<uint4*>(base + s * kStage + b * kBlock + row * 128 + (i & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_any_cta(mapa_shared(smem_u32(&bars->full[s]), leader));
      }
      __syncwarp();
    }
  } else if (warp >= kEpiWarp) {
    group_epilogue<TC, kKind, kRows>(p, tables, bars, tmem_base, crank, warp - kEpiWarp, cluster,
                                     clusters, reinterpret_cast<float*>(base));
  }

  if (parts > 1) {
    // The parts' sums in their order, each CTA for some rows of its columns.
    cluster_sync_all();
    if (cluster < units) {
      const GroupUnit w = group_unit<kKind, kRows>(cluster, p, tables);
      // Four columns of a row per thread, all parts' values on their way at once.  (Only those
      // that are stored are read: see cluster_arrive_relaxed().)
      const int pieces = (w.row_end - w.row) * 32;
      for (int i = part * kThreads + (int)threadIdx.x; i < pieces; i += parts * kThreads) {
        const int col = w.col + (int)rank * 128 + (i & 31) * 4;
        if (col >= p.N) continue;
        const uint32_t at = smem_u32(base) + (uint32_t)i * 16u;
        float4 v[kGroupMaxParts];
#pragma unroll
        for (int j = 0; j < kGroupMaxParts; ++j)
          v[j] = j < parts ? ld_cluster_v4(mapa_shared(at, 2u * j + rank))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
        float sum[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
        for (int j = 1; j < kGroupMaxParts; ++j)
          sum[0] += v[j].x, sum[1] += v[j].y, sum[2] += v[j].z, sum[3] += v[j].w;
        TC* const c = static_cast<TC*>(p.C) + (kWeights ? w.g * p.stride_c : 0) +
                      (long long)(w.row + (i >> 5)) * p.ldc + col;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (col + e < p.N) {
            const float x = p.alpha * sum[e];
            c[e] = from_f32_any<TC>(p.beta == 0.f ? x : fmaf(p.beta, to_f32_any<TC>(c[e]), x));
          }
      }
    }
  }

  // ------------------------------------------------ teardown
  if (warp == 1 && rank == 0 && elect_one()) {
    // Every MMA of the pair has completed before TMEM is freed.
    mma_commit_pair_multicast(smem_u32(&bars->drain), (uint16_t)(1u << leader));
    if (!mbar_wait_bounded(smem_u32(&bars->drain), 0, p.timeout_ns, nullptr))
      raise_fault(p.fault, kFaultDrainWait);
  }
  __syncthreads();
  if (warp == 0 && rank == 0 && elect_one() && bars->abort) {
    // Let the copies in flight land; a stage whose other arrivals are missing
    // makes the wait give up.
    const uint32_t first = issued > (uint32_t)S ? issued - S : 0;
    for (uint32_t it = first; it < issued; ++it) {
      if (!mbar_wait_bounded(smem_u32(&bars->full[it % S]), (it / S) & 1u, p.timeout_ns,
                             nullptr)) {
        raise_fault(p.fault, kFaultDrainWait);
        break;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  // No CTA leaves, nor is TMEM freed, while others may still touch its memory.
  if (bars->abort)
    cluster_arrive_release();
  else
    cluster_arrive_relaxed();
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

template <typename T, typename TC, int kKind, int kRows>
cudaError_t launch_typed(const GroupParams& p, const CUtensorMap* tmM, const CUtensorMap* tmN,
                         const CUtensorMap* tmN16, int pairs, cudaStream_t stream) {
  auto kernel = group_kernel<T, TC, kKind, kRows>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = mx_allow_smem(kernel, Layout<kRows>::kSmem, &done);
  if (e != cudaSuccess) return e;
  return launch_gemm_kernel_clusters(2u << p.log_parts, kernel, dim3(2 * pairs),
                                     dim3(kThreads), Layout<kRows>::kSmem, stream, *tmM, *tmN,
                                     *tmN16, p);
}

template <typename T, typename TC>
cudaError_t launch_kind(const GroupParams& p, const CUtensorMap* a, const CUtensorMap* b,
                        const CUtensorMap* c, int pairs, cudaStream_t s) {
  if (p.kind == kGroupForward)
    return p.tile_rows == 64 ? launch_typed<T, TC, kGroupForward, 64>(p, a, b, c, pairs, s)
                             : launch_typed<T, TC, kGroupForward, 256>(p, a, b, c, pairs, s);
  if (p.kind == kGroupInput)
    return p.tile_rows == 64 ? launch_typed<T, TC, kGroupInput, 64>(p, a, b, c, pairs, s)
                             : launch_typed<T, TC, kGroupInput, 256>(p, a, b, c, pairs, s);
  return launch_typed<T, TC, kGroupWeights, 256>(p, a, b, c, pairs, s);
}

}  // namespace

int group_clusters(int log_parts) {
  static std::atomic<int> known[2][64];
  // (Of one instance: all have the same threads, and nearly the same shared memory.)
  return clusters_at_once(group_kernel<__half, float, kGroupForward, 64>, 2u << log_parts,
                          kThreads, Layout<64>::kSmem, known[log_parts - 1]);
}

cudaError_t launch_group(int dtype, int dtype_c, const GroupParams& p, const CUtensorMap* tmM,
                         const CUtensorMap* tmN, const CUtensorMap* tmN16, int pairs,
                         cudaStream_t stream) {
  if (dtype == 1)
    return dtype_c == 0 ? launch_kind<__half, float>(p, tmM, tmN, tmN16, pairs, stream)
                        : launch_kind<__half, __half>(p, tmM, tmN, tmN16, pairs, stream);
  return dtype_c == 0
             ? launch_kind<__nv_bfloat16, float>(p, tmM, tmN, tmN16, pairs, stream)
             : launch_kind<__nv_bfloat16, __nv_bfloat16>(p, tmM, tmN, tmN16, pairs, stream);
}

}  // namespace dgemm
