// Products of a layer's backward pass on sm_103a tensor cores:
// C = alpha * op(A) . B + beta * C with A FP16 / BF16 and B (K x N) held in a
// microscaled format, blocks of 32 along N.
//
// The scales vary along N, not along the contraction, so they cannot be left
// to a block-scaled MMA: B's codes become 16-bit values on their way into
// shared memory (exact in BF16: 8 significant bits and a power of two) and
// tcgen05.mma.kind::f16 accumulates in FP32.  B is the MMA's M side: a TMEM
// lane is a column of C, and a warp's stores are 32 consecutive columns.
//
// Roles (320 threads): warp 0 loads op(A) by TMA, warp 1 issues the MMAs,
// warps 2-5 drain the accumulators, warps 6-9 read codes and scales and
// write the converted tile (MN-major, 128-byte swizzle).
#include "mx.cuh"

namespace dgemm {
namespace {

constexpr int BM = kMxGradBM, BN = kMxGradBN, BK = kMxGradBK;
constexpr int S = 4;
constexpr int kThreads = 320;
constexpr int kEpiWarps = 4;
constexpr int kConvThreads = 128;
constexpr uint32_t kBlock = 64 * BK * 2;                  // 64 wide, BK deep: 8 KB
constexpr uint32_t kBBytes = BN / 64 * kBlock;            // converted B
constexpr uint32_t kABytes = BM / 64 * kBlock;            // op(A)
constexpr uint32_t kStage = kABytes + kBBytes;
constexpr uint32_t kSmem = S * kStage + 1024 + 256;
constexpr uint32_t kTmemCols = 2 * BM;
static_assert(kTmemCols == 512, "tensor memory holds two accumulators");

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

// 16 codes of one row: 16 bytes (MXINT8) or 8 (MXFP4).
struct Codes16 {
  uint4 w;
  unsigned scale;
};

template <int kFmt, typename T, typename TC, bool kAT>
__global__ void __launch_bounds__(kThreads, 1)
    mx_grad_kernel(const __grid_constant__ CUtensorMap tmA, const MxGradParams p) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char* const base = align_smem_1024(smem_raw);
  Barriers* bars = reinterpret_cast<Barriers*>(base + S * kStage);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int units = p.tiles_m * p.tiles_n;
  const int nk = (p.K + BK - 1) / BK;
  constexpr uint32_t kAb = __is_same(T, __half) ? 0u : 1u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&bars->full[s]), 1 + kConvThreads / 32);
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
  if (warp == 0 && lane == 0) tma_prefetch_desc(&tmA);
  if (warp == 1) tmem_alloc(smem_u32(&bars->tmem_base), kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = bars->tmem_base;
  wait_prior_grids();
  allow_dependent_grids();

  uint32_t issued = 0;
  if (warp == 0) {
    // ------------------------------------------------ op(A)
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
          const uint32_t st = smem_u32(base + s * kStage) + kBBytes;
          mbar_arrive_expect_tx(fb, kABytes);
          if constexpr (kAT) {   // stored K x M: 64-wide blocks of m, one row per k
            for (int j = 0; j < BM / 64; ++j)
              tma_load_2d(st + j * kBlock, &tmA, fb, tm * BM + j * 64, kt * BK);
          } else {               // rows of 64 k
            tma_load_2d(st, &tmA, fb, kt * BK, tm * BM);
          }
          issued = it + 1;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idesc = instr_desc(kAb, BN, BM, 1u, kAT ? 1u : 0u);
      uint32_t it = 0;
      int local = 0;
      bool ok = true;
      for (int u = blockIdx.x; u < units && ok; u += gridDim.x, ++local) {
        const uint32_t b = local & 1;
        ok = role_wait(smem_u32(&bars->acc_empty[b]), ((local >> 1) & 1u) ^ 1u, p.fault,
                       p.timeout_ns, &bars->abort, kFaultTcMmaWait, true);
        if (!ok) break;
        tc_fence_after();
        for (int kt = 0; kt < nk; ++kt, ++it) {
          const uint32_t s = it % S;
          ok = role_wait(smem_u32(&bars->full[s]), (it / S) & 1u, p.fault, p.timeout_ns,
                         &bars->abort, kFaultTcMmaWait, true);
          if (!ok) break;
          tc_fence_after();
          const uint32_t st = smem_u32(base + s * kStage);
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            mma_f16(tmem_base + b * BM, mnmajor_desc(st, k, kBlock),
                    kAT ? mnmajor_desc(st + kBBytes, k, kBlock) : kmajor_desc(st + kBBytes, k),
                    idesc, (kt > 0 || k > 0) ? 1u : 0u);
          mma_commit(smem_u32(&bars->empty[s]));
        }
        if (!ok) break;
        mma_commit(smem_u32(&bars->acc_full[b]));
      }
    }
    __syncwarp();
  } else if (warp < 2 + kEpiWarps) {
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
        store_column32<TC>(r0, static_cast<TC*>(p.C), p.ldc, p.M, p.N, row, col, p.alpha, p.beta);
        store_column32<TC>(r1, static_cast<TC*>(p.C), p.ldc, p.M, p.N, row + 32, col, p.alpha,
                           p.beta);
      }
    }
  } else {
    // ------------------------------------------------ conversion of B
    // Thread t takes 16 columns (t % 8) of rows t / 8 + 16 i of a k-tile.
    const int t = threadIdx.x - 32 * (2 + kEpiWarps);
    const int chunk = t & 7;
    const int row0 = t >> 3;
    constexpr int kRowsPerPass = kConvThreads / 8;
    constexpr int kPasses = BK / kRowsPerPass;
    const int tiles = mx_scale_tiles(p.N);
    uint32_t it = 0;
    bool ok = true;
    for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
      int tn, tm;
      grouped_tile(u, p.tiles_n, p.tiles_m, p.group, tn, tm);
      const int col = tn * BN + chunk * 16;
      for (int kt = 0; kt < nk; ++kt, ++it) {
        Codes16 c[kPasses];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int k = kt * BK + row0 + i * kRowsPerPass;
          c[i].w = make_uint4(0u, 0u, 0u, 0u);
          c[i].scale = 0u;
          if (k < p.K && col < p.N) {   // (a row of codes holds whole groups of 16 columns)
            const unsigned char* src = p.codes + (long long)k * p.ldb;
            if constexpr (kFmt == GEMM_MXFP4) {
              const uint2 w = *reinterpret_cast<const uint2*>(src + col / 2);
              c[i].w.x = w.x;
              c[i].w.y = w.y;
            } else {
              c[i].w = *reinterpret_cast<const uint4*>(src + col);
            }
            c[i].scale = p.sb[mx_scale_offset(k, col >> 5, tiles)];
          }
        }
        const uint32_t s = it % S;
        ok = role_wait_warp(smem_u32(&bars->empty[s]), ((it / S) & 1u) ^ 1u, p.fault,
                            p.timeout_ns, &bars->abort, kFaultTcProducerWait, true);
        if (!ok) break;
        unsigned char* dst = base + s * kStage + (chunk >> 2) * kBlock;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int r = row0 + i * kRowsPerPass;
          const float scale = mx_scale_value(c[i].scale);
          float v[16];
          if constexpr (kFmt == GEMM_MXFP4) {
            float lo[8], hi[8];
            e2m1x8_to_f32(c[i].w.x, lo);
            e2m1x8_to_f32(c[i].w.y, hi);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = lo[j], v[8 + j] = hi[j];
          } else {
            int8x4_to_f32(c[i].w.x, v);
            int8x4_to_f32(c[i].w.y, v + 4);
            int8x4_to_f32(c[i].w.z, v + 8);
            int8x4_to_f32(c[i].w.w, v + 12);
          }
          uint32_t h[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) h[j] = pack2<T>(v[2 * j] * scale, v[2 * j + 1] * scale);
          const int c0 = (chunk & 3) * 2;
          *reinterpret_cast<uint4*>(dst + r * 128 + ((c0 ^ (r & 7)) << 4)) =
              make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(dst + r * 128 + (((c0 + 1) ^ (r & 7)) << 4)) =
              make_uint4(h[4], h[5], h[6], h[7]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->full[s]));
      }
    }
  }

  // ------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 0 && lane == 0 && bars->abort) {
    // Let this CTA's copies in flight land before it exits.  (A stage that
    // the converting warps left out never completes: the wait then gives up.)
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

template <int kFmt, typename T, typename TC, bool kAT>
cudaError_t launch_typed(const MxGradParams& p, const CUtensorMap* tmA, int grid,
                         cudaStream_t stream) {
  auto kernel = mx_grad_kernel<kFmt, T, TC, kAT>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  return launch_gemm_kernel(kernel, dim3(grid), dim3(kThreads), kSmem, stream, *tmA, p);
}

template <int kFmt, typename T>
cudaError_t launch_fmt(const MxGradParams& p, const CUtensorMap* tmA, int grid, cudaStream_t s) {
  if (p.dtype_c == 0)
    return p.op_a ? launch_typed<kFmt, T, float, true>(p, tmA, grid, s)
                  : launch_typed<kFmt, T, float, false>(p, tmA, grid, s);
  return p.op_a ? launch_typed<kFmt, T, T, true>(p, tmA, grid, s)
                : launch_typed<kFmt, T, T, false>(p, tmA, grid, s);
}

}  // namespace

cudaError_t launch_mx_grad(const MxGradParams& p, const CUtensorMap* tmA, int grid,
                           cudaStream_t s) {
  if (p.dtype == 1)
    return p.fmt == GEMM_MXFP4 ? launch_fmt<GEMM_MXFP4, __half>(p, tmA, grid, s)
                               : launch_fmt<GEMM_MXINT8, __half>(p, tmA, grid, s);
  return p.fmt == GEMM_MXFP4 ? launch_fmt<GEMM_MXFP4, __nv_bfloat16>(p, tmA, grid, s)
                             : launch_fmt<GEMM_MXINT8, __nv_bfloat16>(p, tmA, grid, s);
}

}  // namespace dgemm
