// MXFP4 product on sm_103a tensor cores: C = alpha * A . B^T + beta * C with
// A (M x K) and B (N x K) as E2M1 codes and one E8M0 scale per 32 of K.
//
//   c_ij = sum over blocks b of 2^(sa_ib + sb_jb - 254) sum_k a_ik b_jk
//
// tcgen05.mma.kind::mxf4.block_scale forms both sums: codes come from shared
// memory (K-major, 128-byte swizzle), scales from tensor memory, FP32
// accumulation.  B's rows are the MMA's M side: a TMEM lane is a column of C
// and a warp's 32 lanes are 32 consecutive columns, which makes the stores
// of a row contiguous for any alignment of C.
//
// Roles (192 threads): warp 0 loads (TMA for codes, bulk copies for the
// scale tiles, which are contiguous along K), warp 1 issues the copies of
// scales to tensor memory and the MMAs, warps 2-5 drain the accumulators.
#include "mx.cuh"

namespace dgemm {
namespace {

constexpr int BM = kMx4BM, BN = kMx4BN, BK = kMx4BK;
constexpr int S = 5;
constexpr int kThreads = 192;
constexpr int kEpiWarps = 4;
constexpr uint32_t kABytes = BM * BK / 2;     // 16 KB
constexpr uint32_t kBBytes = BN * BK / 2;     // 16 KB
constexpr int kChunks = BK / 128;             // scale tiles along K per stage
constexpr uint32_t kSABytes = BM / 128 * kChunks * kMxTileBytes;
constexpr uint32_t kSBBytes = BN / 128 * kChunks * kMxTileBytes;
constexpr uint32_t kStage = kABytes + kBBytes + kSABytes + kSBBytes;
constexpr uint32_t kSmem = S * kStage + 1024 + 256;
// Tensor memory: two accumulators of BM columns, then scales of two stages
// in turn (4 columns per scale tile).
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScaleCol = 2 * BM;
constexpr uint32_t kScaleStage = 4 * kChunks * (BM / 128 + BN / 128);
static_assert(kScaleCol + 2 * kScaleStage <= kTmemCols, "tensor memory");
static_assert(kStage % 1024 == 0, "stages keep the swizzle's alignment");

struct alignas(8) Barriers {
  uint64_t full[S];
  uint64_t empty[S];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Barriers) <= 256, "barrier block must fit its reserved space");

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    mx4_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
               const Mx4Params p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* const base = align_smem_1024(smem_raw);
  Barriers* bars = reinterpret_cast<Barriers*>(base + S * kStage);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int units = p.tiles_m * p.tiles_n;
  const int nk = (p.K + BK - 1) / BK;
  const int ktiles = mx_scale_tiles(p.K);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&bars->full[s]), 1);
      mbar_init(smem_u32(&bars->empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&bars->acc_full[b]), 1);
      mbar_init(smem_u32(&bars->acc_empty[b]), kEpiWarps);
    }
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) tmem_alloc(smem_u32(&bars->tmem_base), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = bars->tmem_base;
  wait_prior_grids();
  allow_dependent_grids();

  uint32_t issued = 0;
  if (warp == 0) {
    // ------------------------------------------------ loads
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
        int tn, tm;
        grouped_tile(u, p.tiles_n, p.tiles_m, p.group, tn, tm);
        for (int kt = 0; kt < nk; ++kt, ++it) {
          const uint32_t s = it % S;
          ok = role_wait(smem_u32(&bars->empty[s]), ((it / S) & 1u) ^ 1u, p.fault, p.timeout_ns,
                         &bars->abort, kFaultTcProducerWait, true);
          if (!ok) break;
          const uint32_t fb = smem_u32(&bars->full[s]);
          const uint32_t st = smem_u32(base + s * kStage);
          const int chunks = min(kChunks, ktiles - kt * kChunks);
          const uint32_t sbytes = (uint32_t)chunks * kMxTileBytes;
          mbar_arrive_expect_tx(fb, kABytes + kBBytes + 2 * sbytes);
          tma_load_2d(st, &tmB, fb, kt * (BK / 2), tn * BN);
          tma_load_2d(st + kBBytes, &tmA, fb, kt * (BK / 2), tm * BM);
          const long long col = (long long)kt * kChunks;
          bulk_load(st + kBBytes + kABytes, p.sb + ((long long)tn * ktiles + col) * kMxTileBytes,
                    sbytes, fb);
          bulk_load(st + kBBytes + kABytes + kSBBytes,
                    p.sa + ((long long)tm * ktiles + col) * kMxTileBytes, sbytes, fb);
          issued = it + 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    if (lane == 0) {
      uint32_t it = 0;
      int local = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x, ++local) {
        const uint32_t b = local & 1;
        ok = role_wait(smem_u32(&bars->acc_empty[b]), ((local >> 1) & 1u) ^ 1u, p.fault,
                       p.timeout_ns, &bars->abort, kFaultTcMmaWait, true);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem_base + b * BM;
        for (int kt = 0; kt < nk; ++kt, ++it) {
          const uint32_t s = it % S;
          ok = role_wait(smem_u32(&bars->full[s]), (it / S) & 1u, p.fault, p.timeout_ns,
                         &bars->abort, kFaultTcMmaWait, true);
          if (!ok) break;
          tc_fence_after();
          const uint32_t st = smem_u32(base + s * kStage);
          const uint32_t sfb = tmem_base + kScaleCol + (it & 1u) * kScaleStage;
          const uint32_t sfa = sfb + 4 * kChunks;
          const int chunks = min(kChunks, ktiles - kt * kChunks);
          for (int c = 0; c < chunks; ++c) {
            copy_scales(sfb + 4 * c, smem_desc_plain(st + kBBytes + kABytes + c * kMxTileBytes,
                                                     128));
            copy_scales(sfa + 4 * c,
                        smem_desc_plain(st + kBBytes + kABytes + kSBBytes + c * kMxTileBytes, 128));
          }
#pragma unroll
          for (int k = 0; k < BK / 64; ++k) {
            if (k < 2 * chunks)
              mma_mx4(d, kmajor_desc(st, k), kmajor_desc(st + kBBytes, k),
                      instr_desc_mx4(BN, BM, (k & 1) * 2), sfb + 4 * (k >> 1), sfa + 4 * (k >> 1),
                      (kt > 0 || k > 0) ? 1u : 0u);
          }
          mma_commit(smem_u32(&bars->empty[s]));
        }
        if (!ok) break;
        mma_commit(smem_u32(&bars->acc_full[b]));
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue
    const int q = warp & 3;
    int local = 0;
    for (int u = blockIdx.x; u < units; u += gridDim.x, ++local) {
      int tn, tm;
      grouped_tile(u, p.tiles_n, p.tiles_m, p.group, tn, tm);
      const uint32_t b = local & 1;
      if (!role_wait_warp(smem_u32(&bars->acc_full[b]), (local >> 1) & 1u, p.fault, p.timeout_ns,
                          &bars->abort, kFaultTcEpilogueWait, false))
        break;
      tc_fence_after();
      const uint32_t t = tmem_base + ((uint32_t)(q * 32) << 16) + b * BM;
      const int col = tn * BN + q * 32 + lane;
#pragma unroll 1
      for (int c = 0; c < BM / 64; ++c) {
        uint32_t r0[32], r1[32];
        tmem_ld32(t + c * 64, r0);
        tmem_ld32(t + c * 64 + 32, r1);
        tmem_ld_wait(r0, r1);
        if (c == BM / 64 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&bars->acc_empty[b]));
        }
        const int row = tm * BM + c * 64;
        store_column32<T>(r0, static_cast<T*>(p.C), p.ldc, p.M, p.N, row, col, p.alpha, p.beta);
        store_column32<T>(r1, static_cast<T*>(p.C), p.ldc, p.M, p.N, row + 32, col, p.alpha,
                          p.beta);
      }
    }
  }

  // ------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 0 && lane == 0 && bars->abort) {
    // Let this CTA's copies in flight land before it exits.
    const uint32_t first = issued > (uint32_t)S ? issued - S : 0;
    for (uint32_t it = first; it < issued; ++it) {
      if (!mbar_wait_bounded(smem_u32(&bars->full[it % S]), (it / S) & 1u, p.timeout_ns,
                             nullptr)) {
        raise_fault(p.fault, kFaultDrainWait);
        break;
      }
    }
  }
  if (warp == 1) {
    tc_fence_after();
    if (lane == 0) {
      mma_commit(smem_u32(&bars->drain));
      if (!mbar_wait_bounded(smem_u32(&bars->drain), 0, p.timeout_ns, nullptr))
        raise_fault(p.fault, kFaultDrainWait);
    }
    __syncwarp();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <typename T>
cudaError_t launch_typed(const Mx4Params& p, const CUtensorMap* tmA, const CUtensorMap* tmB,
                         int grid, cudaStream_t stream) {
  cudaError_t e =
      cudaFuncSetAttribute(mx4_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_gemm_kernel(mx4_kernel<T>, dim3(grid), dim3(kThreads), kSmem, stream, *tmA, *tmB,
                            p);
}

}  // namespace

cudaError_t launch_mx4(const Mx4Params& p, const CUtensorMap* tmA, const CUtensorMap* tmB,
                       int grid, cudaStream_t stream) {
  if (p.dtype == 0) return launch_typed<float>(p, tmA, tmB, grid, stream);
  if (p.dtype == 1) return launch_typed<__half>(p, tmA, tmB, grid, stream);
  return launch_typed<__nv_bfloat16>(p, tmA, tmB, grid, stream);
}

}  // namespace dgemm
