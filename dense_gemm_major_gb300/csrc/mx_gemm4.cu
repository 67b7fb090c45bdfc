// MXFP4 product on sm_103a tensor cores: C = alpha * A . B^T + beta * C with
// A (M x K) and B (N x K) as E2M1 codes and one E8M0 scale per 32 of K.
//
//   c_ij = sum over blocks b of 2^(sa_ib + sb_jb - 254) sum_k a_ik b_jk
//
// tcgen05.mma.kind::mxf4.block_scale forms both sums: codes come from shared
// memory (K-major, 128-byte swizzle), scales from tensor memory, FP32
// accumulation.
//
// A cluster of two CTAs computes 256 columns x 256 rows of C with
// cta_group::2.  B's rows are the MMA's M side (each CTA loads 128 of them),
// A's its N side (each CTA loads half): a TMEM lane is a column of C and a
// warp's 32 lanes are 32 consecutive columns, which makes the stores of a
// row contiguous for any alignment of C.
//
// Roles (512 threads): warp 12 loads codes and scales by TMA, warp 13 (even
// CTA) issues the MMAs, warps 0-3 write the scales to tensor memory, warps
// 4-11 drain the accumulator.  The scales could go there by tcgen05.cp, but
// its copies take turns with the MMAs in the tensor pipe: 208 against 153 us
// without any at 8192^3.  Tensor memory holds one accumulator of 256 columns
// and the scales of the ring's three stages (two accumulators and two stages
// of scales would not fit): the draining warps take all of it to registers
// before they scale and store, so that the next tile can start.
//
// FP32 results are summed in segments of kMx4SegTerms terms, which the draining
// warps add with rounding: the tensor cores truncate the running sum at each
// step, and where block scales lie so far apart that sums no longer fit 24 bits
// the error grows with their number.  K = 32768, scales over 12 / 16 / 24
// binades: 4.6e-6 / 8.7e-6 / 1.0e-5 of the result's norm in one piece, 5e-7 /
// 1.0e-6 / 1.3e-6 in segments (a plain FP32 product 3e-7); over 8 binades 6e-8,
// over 4, or with a few columns 20 times as large as the others, exact.
// Segments of 1024 / 2048 / 4096 / 8192 terms take 239 / 199 / 180 / 175 us at
// 8192^3, 4096 x 4096 x 16384 119 / 102 / 93 / 89 (in one piece 87).  16-bit
// results round far coarser than either.
//
// Measured: 8192^3 156 us (7.0 PFLOP/s), 4096^3 26.  16384^3 1095 to 1133 (8.0
// to 7.8 PFLOP/s).  At 8192^3 it takes 114 us without its MMAs, 137 without its stores
// and 139 with all of them to one row of C: what stores cost is C's write
// traffic beside the loads, not instructions.  Streaming and write-through
// stores change nothing, whole 128-byte lines per warp 1 to 3 %, stores paced
// over the next tile -2 to -5 % at the largest sizes and +5 % at smaller ones.
#include "mx.cuh"

namespace dgemm {
namespace {

constexpr int BK = kMx4BK;
constexpr int kSegTiles = kMx4SegTerms / BK;
constexpr int S = 3;
constexpr int kThreads = 512;
constexpr int kScaleWarps = 4, kEpiWarp = 4, kEpiWarps = 8, kLoadWarp = 12, kMmaWarp = 13;
// Registers per thread: 128 at launch; after the split 128 threads of scales,
// 128 of loads and MMAs, 256 of draining (128 sums each):
// 72 + 72 + 2 * 184 = 4 * 128.
constexpr int kRegsLaunch = 128, kRegsScale = 72, kRegsIssue = 72, kRegsEpi = 184;
static_assert(kRegsScale + kRegsIssue + 2 * kRegsEpi <= 4 * kRegsLaunch, "register split");
// A stage is two blocks of 256 of K (rows of 128 bytes), each with its part
// of both operands: one barrier round trip of the MMA issuer covers eight
// MMAs.
constexpr int kBlocks = BK / 256;
constexpr uint32_t kHalf = 64 * 128;                     // 64 rows of a block: 8 KB
constexpr uint32_t kBBytes = 2 * kHalf;                  // this CTA's 128 columns of C, a block
constexpr uint32_t kABytes = 2 * kHalf;                  // this CTA's half of the rows
constexpr uint32_t kBlock = kBBytes + kABytes;
constexpr int kChunks = BK / 128;                        // scale tiles along K per stage
constexpr uint32_t kSBytes = kChunks * kMxTileBytes;     // scales of 128 rows: 2 KB
constexpr uint32_t kStage = kBlocks * kBlock + 3 * kSBytes;
constexpr uint32_t kSmem = S * kStage + 1024 + 512;
// Tensor memory columns: the accumulator, then for each stage the scales of
// its four tiles of B (4 columns each) and of A (two row tiles, 8 columns).
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScaleCol = 256;
constexpr uint32_t kScaleStage = 4 * kChunks * 3;
static_assert(kChunks == 4, "16 and 32 columns of scales");
static_assert(kScaleCol + S * kScaleStage <= kTmemCols, "tensor memory");
static_assert(kStage % 1024 == 0, "stages keep the swizzle's alignment");
static_assert(kSmem <= 232448, "shared memory");

struct alignas(8) Barriers {
  uint64_t full[S];     // even CTA: codes of both CTAs loaded, scales of both in TMEM
  uint64_t scales[S];   // scales of this CTA loaded
  uint64_t empty[S];
  uint64_t acc_full;
  uint64_t acc_empty;   // even CTA
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Barriers) <= 512, "barrier block must fit its reserved space");

// kSegments: sums of more than kSegTiles k-tiles in segments.  (Draining a
// segment to add it takes longer than draining all columns at once: 7.5
// against 7.0 us at 1000 x 1030 x 777.)
template <typename T, bool kSegments>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mx4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
               const Mx4Params p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* const base = align_smem_1024(smem_raw);
  Barriers* bars = reinterpret_cast<Barriers*>(base + S * kStage);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();   // 0: issues the MMAs
  const int npairs = gridDim.x >> 1;
  const int nk = (p.K + BK - 1) / BK;
  const int ktiles = mx_scale_tiles(p.K);
  const MxSchedule& sc = p.sched;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&bars->full[s]), 1 + 2 * kScaleWarps);
      mbar_init(smem_u32(&bars->scales[s]), 1);
      mbar_init(smem_u32(&bars->empty[s]), 1);
    }
    mbar_init(smem_u32(&bars->acc_full), 1);
    mbar_init(smem_u32(&bars->acc_empty), 2 * kEpiWarps);
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
  }
  if (warp == kMmaWarp) tmem_alloc_pair(smem_u32(&bars->tmem_base), kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = bars->tmem_base;
  wait_prior_grids();
  allow_dependent_grids();

  uint32_t issued = 0;
  if (warp < kScaleWarps) {
    // ------------------------------------------------ scales to tensor memory (both CTAs)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsScale));
    // Lane l of warp q writes lane 32 q + l: row l of a tile, 16 bytes, is its
    // four columns there, the same in all four quarters.
    const uint32_t t = tmem_base + ((uint32_t)(warp * 32) << 16) + kScaleCol;
    RingPos<S> pos;
    bool ok = true;
    for (int u = blockIdx.x >> 1; u < sc.units && ok; u += npairs) {
      const MxUnit w = mx_unit(u, sc, nk);
      if (w.row0 >= p.M) continue;
      for (int kt = w.kb; kt < w.ke; ++kt, pos.next()) {
        const uint32_t s = pos.slot;
        // (The loads were issued after the MMAs on this stage had finished, so
        // its columns may be overwritten.)
        ok = role_wait_lanes(smem_u32(&bars->scales[s]), pos.parity, p.fault, p.timeout_ns,
                             &bars->abort, kFaultTcProducerWait);
        if (!ok) break;
        const uint4* tile =
            reinterpret_cast<const uint4*>(base + s * kStage + kBlocks * kBlock) + lane;
        constexpr int kTile = kMxTileBytes / 16;
        uint32_t rb[16], ra[32];
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const uint4 x = tile[c * kTile];
          const uint4 y = tile[(kChunks + c) * kTile], z = tile[(2 * kChunks + c) * kTile];
          rb[4 * c] = x.x, rb[4 * c + 1] = x.y, rb[4 * c + 2] = x.z, rb[4 * c + 3] = x.w;
          ra[8 * c] = y.x, ra[8 * c + 1] = y.y, ra[8 * c + 2] = y.z, ra[8 * c + 3] = y.w;
          ra[8 * c + 4] = z.x, ra[8 * c + 5] = z.y, ra[8 * c + 6] = z.z, ra[8 * c + 7] = z.w;
        }
        tmem_st16(t + s * kScaleStage, rb);
        tmem_st32(t + s * kScaleStage + 4 * kChunks, ra);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_any_cta(mapa_shared(smem_u32(&bars->full[s]), 0));
      }
    }
    __syncwarp();
  } else if (warp >= kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == kLoadWarp && elect_one()) {
      // ---------------------------------------------- loads (both CTAs)
      RingPos<S> pos;
      uint32_t it = 0;
      bool ok = true;
      for (int u = blockIdx.x >> 1; u < sc.units && ok; u += npairs) {
        const MxUnit w = mx_unit(u, sc, nk);
        if (w.row0 >= p.M) continue;
        const int halves = w.rows / 128;            // 64-row boxes of A per CTA
        const int row = w.row0 + (int)rank * (w.rows / 2);
        const int ct = w.tn * 2 + (int)rank;
        for (int kt = w.kb; kt < w.ke; ++kt, ++it, pos.next()) {
          const uint32_t s = pos.slot;
          ok = role_wait(smem_u32(&bars->empty[s]), pos.parity ^ 1u, p.fault, p.timeout_ns,
                         &bars->abort, kFaultTcProducerWait, true);
          if (!ok) break;
          const uint32_t fb = mapa_shared(smem_u32(&bars->full[s]), 0);
          if (rank == 0)
            mbar_arrive_expect_tx(smem_u32(&bars->full[s]),
                                  2u * kBlocks * (kBBytes + halves * kHalf));
          const uint32_t st = smem_u32(base + s * kStage);
          for (int b = 0; b < kBlocks; ++b) {
            const int x = kt * (BK / 2) + b * 128;
            tma_load_2d_pair(st + b * kBlock, &tmB, fb, x, ct * 128);
            for (int j = 0; j < halves; ++j)
              tma_load_2d_pair(st + b * kBlock + kBBytes + j * kHalf, &tmA, fb, x, row + j * 64);
          }
          const uint32_t ss = st + kBlocks * kBlock;
          const int x = kt * (int)(kSBytes / 8);
          const uint32_t sb = smem_u32(&bars->scales[s]);
          mbar_arrive_expect_tx(sb, (1 + halves) * kSBytes);
          tma_load_2d(ss, &tmSB, sb, x, ct);
          // The scales of all of the tile's rows of C, in both CTAs.
          for (int j = 0; j < halves; ++j)
            tma_load_2d(ss + (1 + j) * kSBytes, &tmSA, sb, x, w.row0 / 128 + j);
          issued = it + 1;
        }
      }
    } else if (warp == kMmaWarp && rank == 0 && elect_one()) {
      // ---------------------------------------------- MMA issuer (even CTA)
      // The barrier of the next stage is tried before this stage's MMAs are
      // issued: a try takes over 100 cycles to answer.
      RingPos<S> pos;
      bool ready = false;
      uint32_t local = 0;
      bool ok = true;
      for (int u = blockIdx.x >> 1; u < sc.units && ok; u += npairs) {
        const MxUnit w = mx_unit(u, sc, nk);
        if (w.row0 >= p.M) continue;
        const uint32_t idesc = instr_desc_mx4(256, (uint32_t)w.rows, 0);
        const uint32_t idesc2 = instr_desc_mx4(256, (uint32_t)w.rows, 2);
        int k0 = w.kb;
        do {
          const int k1 = kSegments ? min(k0 + kSegTiles, w.ke) : w.ke;
          ok = role_wait(smem_u32(&bars->acc_empty), (local & 1u) ^ 1u, p.fault, p.timeout_ns,
                         &bars->abort, kFaultTcMmaWait, true);
          if (!ok) break;
          tc_fence_after();
          for (int kt = k0; kt < k1; ++kt) {
            const uint32_t s = pos.slot;
            const uint32_t st = smem_u32(base + s * kStage);
            ok = ready || role_wait(smem_u32(&bars->full[s]), pos.parity, p.fault, p.timeout_ns,
                                    &bars->abort, kFaultTcMmaWait, true);
            if (!ok) break;
            tc_fence_after();
            pos.next();
            ready = mbar_try_wait(smem_u32(&bars->full[pos.slot]), pos.parity);
            const uint32_t blo = desc_lo(st, 16), alo = desc_lo(st + kBBytes, 16);
            const uint32_t sfb = tmem_base + kScaleCol + s * kScaleStage;
            const uint32_t sfa = sfb + 4 * kChunks;
            const int chunks = min(kChunks, ktiles - kt * kChunks);
#pragma unroll
            for (int k = 0; k < BK / 64; ++k) {
              if (k < 2 * chunks) {
                const uint32_t off = ((k >> 2) * kBlock + (k & 3) * 32) >> 4;
                mma_mx4_pair(tmem_base, blo + off, alo + off, (k & 1) ? idesc2 : idesc,
                             sfb + 4 * (k >> 1), sfa + 8 * (k >> 1),
                             (kt > k0 || k > 0) ? 1u : 0u);
              }
            }
            mma_commit_pair_multicast(smem_u32(&bars->empty[s]), 0x3);
          }
          if (!ok) break;
          mma_commit_pair_multicast(smem_u32(&bars->acc_full), 0x3);
          ++local;
          k0 = k1;
        } while (kSegments && k0 < w.ke);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue (both CTAs)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    // Warp: TMEM lanes 32 q .. 32 q + 31 (columns of C), half of the rows.
    const int q = warp & 3;
    const int half = (warp - kEpiWarp) >> 2;
    const bool pairs = (reinterpret_cast<uintptr_t>(p.C) & 3u) == 0 && ((p.ldc | p.N) & 1) == 0;
    uint32_t local = 0;
    bool ok = true;
    for (int u = blockIdx.x >> 1; u < sc.units && ok; u += npairs) {
      const MxUnit w = mx_unit(u, sc, nk);
      if (w.row0 >= p.M) continue;
      const int chunks = w.rows / 64;      // of 32 rows, this warp's share
      const int first = half * (w.rows / 2);
      const uint32_t t = tmem_base + ((uint32_t)(q * 32) << 16) + first;
      uint32_t r[4][32];
      if constexpr (kSegments) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int j = 0; j < 32; ++j) r[c][j] = 0x80000000u;   // -0
        }
      }
      int k0 = w.kb;
      do {
        ok = role_wait_lanes(smem_u32(&bars->acc_full), local & 1u, p.fault, p.timeout_ns,
                             &bars->abort, kFaultTcEpilogueWait, false, false);
        if (!ok) break;
        tc_fence_after();
        if constexpr (!kSegments) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (c < chunks) tmem_ld32(t + c * 32, r[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld_wait32(r[c]);
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (c < 2 * chunks) {
              uint32_t x[16];
              tmem_ld16(t + c * 16, x);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                uint32_t& sum = r[c / 2][(c & 1) * 16 + j];
                sum = __float_as_uint(__uint_as_float(sum) + __uint_as_float(x[j]));
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_any_cta(mapa_shared(smem_u32(&bars->acc_empty), 0));
        ++local;
        k0 += kSegTiles;
      } while (kSegments && k0 < w.ke);
      if (!ok) break;
      const int col = w.tn * 256 + (int)rank * 128 + q * 32 + lane;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c < chunks) {
          const int row = w.row0 + first + c * 32;
          const float* v = reinterpret_cast<const float*>(r[c]);
          if (sc.slices == 1)
            store_piece<T>(v, static_cast<T*>(p.C), p.ldc, p.M, p.N, row, col, pairs, p.alpha,
                           p.beta);
          else if (col < p.N)
            store_rows32<float>(v, p.ws + ((long long)w.slice * p.M + row) * p.ldw + col, p.ldw,
                                p.M - row, 1.f, 0.f);
        }
      }
    }
  }

  // ------------------------------------------------ teardown
  if (warp == kMmaWarp && rank == 0 && elect_one()) {
    mma_commit_pair_multicast(smem_u32(&bars->drain), 0x1);
    if (!mbar_wait_bounded(smem_u32(&bars->drain), 0, p.timeout_ns, nullptr))
      raise_fault(p.fault, kFaultDrainWait);
  }
  if (warp == kLoadWarp && elect_one() && bars->abort) {
    // Let the loads in flight land: this CTA's scales, and (even CTA) both
    // CTAs' codes on full[], whose arrivals by the warps of scales may be
    // missing; the wait then gives up.
    const uint32_t first = issued > (uint32_t)S ? issued - S : 0;
    for (uint32_t it = first; it < issued; ++it) {
      const uint32_t s = it % S, ph = (it / S) & 1u;
      bool ok = mbar_wait_bounded(smem_u32(&bars->scales[s]), ph, p.timeout_ns, nullptr);
      if (ok && rank == 0)
        ok = mbar_wait_bounded(smem_u32(&bars->full[s]), ph, p.timeout_ns, nullptr);
      if (!ok) {
        raise_fault(p.fault, kFaultDrainWait);
        break;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // neither CTA leaves while the pair may still touch its memory
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

template <typename T, bool kSegments>
cudaError_t launch_kernel(const Mx4Params& p, const CUtensorMap* tmA, const CUtensorMap* tmB,
                         const CUtensorMap* tmSA, const CUtensorMap* tmSB, int pairs,
                         cudaStream_t stream) {
  // The register split needs kRegsLaunch registers a thread at launch: with
  // fewer, its setmaxnreg.inc would wait for ever.
  static const bool fits = [] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, mx4_kernel<T, kSegments>) == cudaSuccess && a.numRegs == kRegsLaunch;
  }();
  if (!fits) return cudaErrorInvalidConfiguration;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = mx_allow_smem(mx4_kernel<T, kSegments>, kSmem, &done);
  if (e != cudaSuccess) return e;
  return launch_gemm_kernel(mx4_kernel<T, kSegments>, dim3(2 * pairs), dim3(kThreads), kSmem, stream, *tmA,
                            *tmB, *tmSA, *tmSB, p);
}

template <typename T>
cudaError_t launch_typed(const Mx4Params& p, const CUtensorMap* tmA, const CUtensorMap* tmB,
                         const CUtensorMap* tmSA, const CUtensorMap* tmSB, int pairs,
                         cudaStream_t stream) {
  if constexpr (sizeof(T) == 4) {
    const int nk = (p.K + BK - 1) / BK;
    if ((nk + p.sched.slices - 1) / p.sched.slices > kSegTiles)
      return launch_kernel<T, true>(p, tmA, tmB, tmSA, tmSB, pairs, stream);
  }
  return launch_kernel<T, false>(p, tmA, tmB, tmSA, tmSB, pairs, stream);
}

}  // namespace

cudaError_t launch_mx4(const Mx4Params& p, const CUtensorMap* tmA, const CUtensorMap* tmB,
                       const CUtensorMap* tmSA, const CUtensorMap* tmSB, int pairs,
                       cudaStream_t stream) {
  if (p.dtype == 0) return launch_typed<float>(p, tmA, tmB, tmSA, tmSB, pairs, stream);
  if (p.dtype == 1) return launch_typed<__half>(p, tmA, tmB, tmSA, tmSB, pairs, stream);
  return launch_typed<__nv_bfloat16>(p, tmA, tmB, tmSA, tmSB, pairs, stream);
}

}  // namespace dgemm
