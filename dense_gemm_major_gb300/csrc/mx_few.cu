// C = alpha * A . B^T + beta * C for up to 64 rows of A (decoding, small
// batches), B (N x K) in MXFP4; A either in MXFP4 or, up to kMx4FewRawRows
// rows of moderate length, a 16- or 32-bit array that is quantised to MXFP4 on
// the way, in the same launch.
//
// What bounds it is reading B once (N K 17 / 32 bytes) and, for a few rows,
// latency.  B's rows are the M side of tcgen05.mma.kind::mxf4 (128 columns of
// C per CTA) and A's its N side (16 to 64), so that no tile is wasted on
// rows that do not exist.  So that B's bytes travel to all SMs at once, the
// CTAs of a cluster share a tile's K; they add their FP32 partial tiles
// through distributed shared memory in rank order, so results are
// reproducible and there is no workspace and no second launch.
//
// Measured at N = K = 4096, back to back: 1 row 4.9 us, 8 5.1, 33 7.8 (a cold
// read of B's 8.9 MB alone takes 1.3 us; launch, tensor memory, barriers and
// the two cluster barriers are the most of the rest).
//
// Roles (320 threads): warp 0 loads codes (TMA) and scales (bulk copies),
// warp 1 issues scale copies and MMAs, warps 2-9 quantise A where it comes
// unquantised, and warps 2-5 then drain the accumulator.
#include "mx.cuh"

namespace dgemm {
namespace {

constexpr int BN = 128, BK = 256;
constexpr int kThreads = 320;
constexpr int kWorkWarp = 2;
constexpr int kChunks = BK / 128;                        // scale tiles along K per stage
constexpr uint32_t kBBytes = BN * BK / 2;                // 16 KB
constexpr uint32_t kSBytes = kChunks * kMxTileBytes;     // 1 KB

// FP32 results: the tensor cores truncate the running sum at each step, and
// where block scales lie so far apart that sums no longer fit 24 bits the
// error grows with their number (over 32768 terms 1e-5 of the result's norm with
// scales over 24 binades; see mx_gemm4.cu).  So a sum of
// at most kMx4SegTerms terms is formed in the accumulator, and such sums are
// added with rounding in other columns of tensor memory.
constexpr int kSegTiles = kMx4SegTerms / BK;

// MT: rows of A that the MMA computes; kSums: with columns for the sums of
// segments.
template <int MT, bool kSums>
struct Layout {
  // Two CTAs fit an SM, so that one's MMAs and scale copies run beside the
  // other's: 64 x 8192 x 8192 took 14 us with one of twice the stages.
  static constexpr int kStages = 4;
  // The quantising warps work in groups, each on stages of its own, so that
  // several stages' loads of A are in flight at once.  Stages are a multiple
  // of groups: a slot's stages all fall to one group, which therefore never
  // waits for a phase whose predecessor it has not seen.
  static constexpr int kGroups = 2;
  static constexpr int kGroupWarps = 8 / kGroups;
  static_assert(kStages % kGroups == 0, "one group per slot");
  static constexpr uint32_t kABytes = MT * BK / 2;
  static constexpr uint32_t kStage = (kBBytes + kABytes + 2 * kSBytes + 1023) / 1024 * 1024;
  static constexpr uint32_t kSmem = kStages * kStage + 1024 + 256;
  // Tensor memory: the accumulator, the scales of two stages, the sums.
  static constexpr uint32_t kScaleCol = MT;
  static constexpr uint32_t kSumCol = kScaleCol + 4 * 4 * kChunks;
  static constexpr uint32_t kUsedCols = kSumCol + (kSums ? MT : 0);
  static constexpr uint32_t kTmemCols = kUsedCols <= 64 ? 64 : (kUsedCols <= 128 ? 128 : 256);
  static_assert(2 * kTmemCols <= 512, "tensor memory of two CTAs");
  static_assert(MT * BN * 4 <= kStages * kStage, "partial tiles reuse the ring");
  static_assert(2 * (kSmem + 1024) <= 233472, "two CTAs per SM");
};

template <int S>
struct alignas(8) Barriers {
  uint64_t full[S];     // loaded, and A quantised
  uint64_t empty[S];
  uint64_t acc_full;
  uint64_t acc_empty;   // a segment's sum has been taken
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

// 64-deep block-scaled MMA step, and the copy of a 512-byte tile of scales
// to 4 TMEM columns (all four lane quarters), on one CTA.
__device__ __forceinline__ void mma_mx4(uint32_t d_tmem, uint32_t alo, uint32_t blo,
                                        uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %7, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %4, [%5], "
      "[%6], p;\n\t}" ::"r"(d_tmem),
      "r"(alo), "r"(blo), "r"(kDescHi128B), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t lo) {
  asm volatile(
      "{\n\t.reg .b64 s;\n\tmov.b64 s, {%1, %2};\n\t"
      "tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], s;\n\t}" ::"r"(taddr),
      "r"(lo), "r"(kDescHiPlain)
      : "memory");
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

// One element of C.
template <typename T>
__device__ __forceinline__ void store_scaled(T* c, float sum, float alpha, float beta) {
  float v = alpha * sum;
  if (beta != 0.f) v = fmaf(beta, to_f32_any<T>(*c), v);
  *c = from_f32_any<T>(v);
}

// kRaw: A is p.X, an array of T.  kSegments: sums of more than kSegTiles stages
// in segments.
template <int MT, typename T, bool kRaw, bool kSegments>
__global__ void __launch_bounds__(kThreads, 2)
    mx4_few_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const Mx4FewParams p) {
  using L = Layout<MT, kSegments>;
  constexpr int S = L::kStages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* const base = align_smem_1024(smem_raw);
  auto* bars = reinterpret_cast<Barriers<S>*>(base + S * L::kStage);
  static_assert(sizeof(Barriers<S>) <= 256, "barrier block must fit its reserved space");
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int tn = blockIdx.x / p.split;
  const int rank = blockIdx.x - tn * p.split;
  const int nk = (p.K + BK - 1) / BK;
  const int kb = (int)((long long)rank * nk / p.split);
  const int ke = (int)((long long)(rank + 1) * nk / p.split);
  const int ktiles = mx_scale_tiles(p.K);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&bars->full[s]), 1 + (kRaw ? L::kGroupWarps : 0));
      mbar_init(smem_u32(&bars->empty[s]), 1);
    }
    mbar_init(smem_u32(&bars->acc_full), 1);
    mbar_init(smem_u32(&bars->acc_empty), 4);
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    if (!kRaw) tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) tmem_alloc(smem_u32(&bars->tmem_base), L::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = bars->tmem_base;
  wait_prior_grids();
  allow_dependent_grids();

  uint32_t issued = 0;
  if (warp == 0) {
    // ------------------------------------------------ loads
    if (elect_one()) {
      for (int kt = kb; kt < ke; ++kt) {
        const uint32_t it = (uint32_t)(kt - kb), s = it % S;
        if (!role_wait(smem_u32(&bars->empty[s]), ((it / S) & 1u) ^ 1u, p.fault, p.timeout_ns,
                       &bars->abort, kFaultTcProducerWait, true))
          break;
        const uint32_t fb = smem_u32(&bars->full[s]);
        const uint32_t st = smem_u32(base + s * L::kStage);
        const uint32_t sbytes = (uint32_t)min(kChunks, ktiles - kt * kChunks) * kMxTileBytes;
        const uint32_t ss = st + kBBytes + L::kABytes;
        mbar_arrive_expect_tx(fb, kBBytes + sbytes + (kRaw ? 0u : L::kABytes + sbytes));
        tma_load_2d(st, &tmB, fb, kt * (BK / 2), tn * BN);
        const long long col = (long long)kt * kChunks;
        bulk_load(ss, p.sb + ((long long)tn * ktiles + col) * kMxTileBytes, sbytes, fb);
        if constexpr (!kRaw) {
          tma_load_2d(st + kBBytes, &tmA, fb, kt * (BK / 2), 0);
          bulk_load(ss + kSBytes, p.sa + col * kMxTileBytes, sbytes, fb);
        }
        issued = it + 1;
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------ MMA issuer
    if (elect_one()) {
      bool ok = true;
      for (int kt = kb; kt < ke; ++kt) {
        const uint32_t it = (uint32_t)(kt - kb), s = it % S;
        const bool starts = kSegments ? it % kSegTiles == 0 : it == 0;   // a segment
        if (kSegments && starts && it > 0) {
          mma_commit(smem_u32(&bars->acc_full));
          ok = role_wait(smem_u32(&bars->acc_empty), (it / kSegTiles - 1) & 1u, p.fault,
                         p.timeout_ns, &bars->abort, kFaultTcMmaWait, true);
          if (!ok) break;
        }
        ok = role_wait(smem_u32(&bars->full[s]), (it / S) & 1u, p.fault, p.timeout_ns,
                       &bars->abort, kFaultTcMmaWait, true);
        if (!ok) break;
        tc_fence_after();
        const uint32_t st = smem_u32(base + s * L::kStage);
        const uint32_t sx = st + kBBytes, ss = sx + L::kABytes;
        const uint32_t sfw = tmem_base + L::kScaleCol + (it & 1u) * 8 * kChunks;
        const uint32_t sfx = sfw + 4 * kChunks;
        const uint32_t blo = desc_lo(st, 16), alo = desc_lo(sx, 16);
        const int chunks = min(kChunks, ktiles - kt * kChunks);
        for (int c = 0; c < chunks; ++c) {
          copy_scales(sfw + 4 * c, desc_lo(ss + c * kMxTileBytes, 0));
          copy_scales(sfx + 4 * c, desc_lo(ss + kSBytes + c * kMxTileBytes, 0));
        }
#pragma unroll
        for (int k = 0; k < BK / 64; ++k)
          if (k < 2 * chunks)
            mma_mx4(tmem_base, blo + 2 * k, alo + 2 * k,
                    instr_desc_mx4(BN, MT, (k & 1) * 2), sfw + 4 * (k >> 1), sfx + 4 * (k >> 1),
                    (!starts || k > 0) ? 1u : 0u);
        mma_commit(smem_u32(&bars->empty[s]));
      }
      if (ok) mma_commit(smem_u32(&bars->acc_full));
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ quantisation, then the epilogue
    const int v = (warp - kWorkWarp) % L::kGroupWarps;
    bool ok = true;
    // Takes the accumulator of segment `taken`, not the last one, by warps 2-5.
    uint32_t taken = 0;
    const uint32_t lanes = tmem_base + ((uint32_t)((warp & 3) * 32) << 16);
    auto take_segment = [&] {
      ok = role_wait_lanes(smem_u32(&bars->acc_full), taken & 1u, p.fault, p.timeout_ns,
                           &bars->abort, kFaultTcEpilogueWait);
      if (!ok) return;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < MT / 16 && c * 16 < p.M; ++c) {
        uint32_t r[16];
        tmem_ld16(lanes + c * 16, r);
        if (taken > 0) {
          uint32_t sum[16];
          tmem_ld16(lanes + L::kSumCol + c * 16, sum);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            r[j] = __float_as_uint(__uint_as_float(r[j]) + __uint_as_float(sum[j]));
        }
        tmem_st16(lanes + L::kSumCol + c * 16, r);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->acc_empty));
      ++taken;
    };
    for (int kt = kb + (warp - kWorkWarp) / L::kGroupWarps; kRaw && kt < ke; kt += L::kGroups) {
      const uint32_t it = (uint32_t)(kt - kb), s = it % S;
      // (Every stage before this segment is, or will be, quantised without
      // waiting for this warp.)
      if (kSegments && warp < kWorkWarp + 4)
        while (ok && (taken + 1) * kSegTiles <= it) take_segment();
      if (!ok) break;
      ok = role_wait_lanes(smem_u32(&bars->empty[s]), ((it / S) & 1u) ^ 1u, p.fault, p.timeout_ns,
                           &bars->abort, kFaultTcProducerWait);
      if (!ok) break;
      unsigned char* sx = base + s * L::kStage + kBBytes;
      unsigned char* ss = sx + L::kABytes + kSBytes;
      // A lane takes whole blocks: 8 of a row per stage, 16 bytes of codes
      // each, which is one chunk of the swizzled row.  (Four lanes to a block,
      // as in the kernel that only quantises, took 4 to 8 % longer.  Rows past
      // M stay as they are: they only reach columns of the accumulator that
      // are not stored.)
#pragma unroll 2
      for (int i = v * 32 + lane; i < 8 * p.M; i += 32 * L::kGroupWarps) {
        const int m = i >> 3, b = i & 7;
        const int k0 = kt * BK + b * kMxBlock;
        const T* src = static_cast<const T*>(p.X) + (long long)m * p.ldx + k0;
        float x[4][8];
        if (p.vec && k0 + kMxBlock <= p.K) {
#pragma unroll
          for (int g = 0; g < 4; ++g) load8<T>(src + 8 * g, x[g]);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j >> 3][j & 7] = k0 + j < p.K ? to_f32_any<T>(src[j]) : 0.f;
        }
        unsigned amax = 0;
#pragma unroll
        for (int j = 0; j < 32; ++j) amax = max(amax, abs_bits(x[j >> 3][j & 7]));
        const unsigned sb = mx_scale_byte<GEMM_MXFP4>(amax);
        const float inv = mx_inverse_scale(sb);
        unsigned q[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[g][j] *= inv;
          q[g] = sb == 255u ? 0u : e2m1x8(x[g]);
        }
        *reinterpret_cast<uint4*>(sx + m * 128 + ((b ^ (m & 7)) << 4)) =
            make_uint4(q[0], q[1], q[2], q[3]);
        ss[(b >> 2) * kMxTileBytes + (m & 31) * 16 + (m >> 5) * 4 + (b & 3)] = (unsigned char)sb;
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars->full[s]));
    }
    if (warp < kWorkWarp + 4) {
      const int q = warp & 3;
      if (kSegments)
        while (ok && (int)(taken + 1) * kSegTiles < ke - kb) take_segment();
      if (ke > kb)
        ok = ok && role_wait_lanes(smem_u32(&bars->acc_full), taken & 1u, p.fault, p.timeout_ns,
                                   &bars->abort, kFaultTcEpilogueWait);
      tc_fence_after();
      const int col = q * 32 + lane;           // within the tile
#pragma unroll 1
      for (int c = 0; c < MT / 16; ++c) {
        if (c * 16 >= p.M) break;
        uint32_t r[16];
        tmem_ld16(lanes + c * 16, r);
        if (kSegments && taken > 0) {
          uint32_t sum[16];
          tmem_ld16(lanes + L::kSumCol + c * 16, sum);
#pragma unroll
          for (int j = 0; j < 16; ++j)
            r[j] = __float_as_uint(__uint_as_float(sum[j]) + __uint_as_float(r[j]));
        }
        if (p.split > 1) {
          // The partial tile, row-major, where the ring was.
          float* part = reinterpret_cast<float*>(base) + c * 16 * BN + col;
#pragma unroll
          for (int j = 0; j < 16; ++j) part[j * BN] = ke > kb ? __uint_as_float(r[j]) : 0.f;
        } else if (tn * BN + col < p.N) {
          T* y = static_cast<T*>(p.C) + (long long)(c * 16) * p.ldc + tn * BN + col;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c * 16 + j < p.M)
              store_scaled<T>(y + j * p.ldc, __uint_as_float(r[j]), p.alpha, p.beta);
        }
      }
    }
  }
  if (p.split > 1) {
    // ------------------------------------------------ sum of the cluster's partial tiles
    cluster_sync_all();
    // This CTA adds up BN / split of the columns, four of a row per thread, all
    // partial tiles' values on their way at once (33 x 4096 x 4096 8.9 -> 8.6 us
    // against one value after the other).
    constexpr int kMaxSplit = 8;
    const int share = BN / p.split / 4;
    for (int i = threadIdx.x; i < share * p.M; i += kThreads) {
      const int m = i / share;
      const int col = (rank * share + (i - m * share)) * 4;
      const uint32_t at = smem_u32(base) + (uint32_t)(m * BN + col) * 4u;
      float4 v[kMaxSplit];
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r)
        v[r] = r < p.split ? ld_cluster_v4(mapa_shared(at, (uint32_t)r))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
      float sum[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int r = 1; r < kMaxSplit; ++r) {
        sum[0] += v[r].x;
        sum[1] += v[r].y;
        sum[2] += v[r].z;
        sum[3] += v[r].w;
      }
      T* c = static_cast<T*>(p.C) + (long long)m * p.ldc + tn * BN + col;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (tn * BN + col + j < p.N) store_scaled<T>(c + j, sum[j], p.alpha, p.beta);
    }
    cluster_sync_all();   // no CTA leaves while others read its partial tile
  }

  // ------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 0 && elect_one() && bars->abort) {
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
    if (elect_one() && bars->abort) {
      // (Otherwise acc_full has shown every MMA to be done.)
      mma_commit(smem_u32(&bars->drain));
      if (!mbar_wait_bounded(smem_u32(&bars->drain), 0, p.timeout_ns, nullptr))
        raise_fault(p.fault, kFaultDrainWait);
    }
    __syncwarp();
    tmem_dealloc(tmem_base, L::kTmemCols);
  }
}

template <int MT, typename T, bool kRaw, bool kSegments>
cudaError_t launch_kernel(const Mx4FewParams& p, const CUtensorMap* tmA, const CUtensorMap* tmB,
                          cudaStream_t stream) {
  auto kernel = mx4_few_kernel<MT, T, kRaw, kSegments>;
  constexpr int smem = Layout<MT, kSegments>::kSmem;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = mx_allow_smem(kernel, smem, &done);
  if (e != cudaSuccess) return e;
  const int tiles = (p.N + BN - 1) / BN;
  return launch_gemm_kernel_clusters((unsigned)p.split, kernel, dim3((unsigned)(tiles * p.split)),
                                     dim3(kThreads), smem, stream, *tmA, *tmB, p);
}

template <int MT, typename T, bool kRaw>
cudaError_t launch_typed(const Mx4FewParams& p, const CUtensorMap* tmA, const CUtensorMap* tmB,
                         cudaStream_t stream) {
  if constexpr (sizeof(T) == 4) {
    const int nk = (p.K + BK - 1) / BK;
    if ((nk + p.split - 1) / p.split > kSegTiles)
      return launch_kernel<MT, T, kRaw, true>(p, tmA, tmB, stream);
  }
  return launch_kernel<MT, T, kRaw, false>(p, tmA, tmB, stream);
}

template <typename T>
cudaError_t launch_rows(const Mx4FewParams& p, const CUtensorMap* a, const CUtensorMap* b,
                        cudaStream_t s) {
  const bool raw = p.X != nullptr;
  switch (mx4_few_tile(p.M)) {
    case 16:
      return raw ? launch_typed<16, T, true>(p, a, b, s) : launch_typed<16, T, false>(p, a, b, s);
    case 32:
      return raw ? launch_typed<32, T, true>(p, a, b, s) : launch_typed<32, T, false>(p, a, b, s);
    default:
      return raw ? launch_typed<64, T, true>(p, a, b, s) : launch_typed<64, T, false>(p, a, b, s);
  }
}

}  // namespace

cudaError_t launch_mx4_few(const Mx4FewParams& p, const CUtensorMap* tmA, const CUtensorMap* tmB,
                           cudaStream_t stream) {
  if (p.dtype == 0) return launch_rows<float>(p, tmA, tmB, stream);
  if (p.dtype == 1) return launch_rows<__half>(p, tmA, tmB, stream);
  return launch_rows<__nv_bfloat16>(p, tmA, tmB, stream);
}

}  // namespace dgemm
