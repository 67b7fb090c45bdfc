// Products of a layer's backward pass on sm_103a tensor cores:
// C = alpha * op(A) . B + beta * C with A FP16 / BF16 and B (K x N) held in a
// microscaled format, blocks of 32 along N.
//
// The scales vary along N, not along the contraction, so they cannot be left
// to a block-scaled MMA: B's codes become 16-bit values inside the kernel
// (exact in BF16: at most 8 significant bits and a power of two) and
// tcgen05.mma.kind::f16 accumulates in FP32.
//
// A cluster of two CTAs computes 256 columns x 256 rows of C with
// cta_group::2.  B is the MMA's M side (each CTA converts its own 128
// columns), op(A) its N side (each CTA loads half of the rows): a TMEM lane
// is a column of C, so that a warp stores 32 consecutive columns of a row,
// whatever C's alignment, and B, which costs instructions, is the operand
// that no CTA touches twice per tile.
//
// Roles (640 threads): warp 0 loads op(A) by TMA, warp 1 issues the MMAs
// (even CTA), warp 2 loads the codes (TMA) and tiles of scales into a ring of
// their own, ahead of the MMAs' ring, warps 4-11 convert, warps 12-19 drain
// the accumulators.
//
// FP32 sums.  The MMA truncates the running sum at every 16-deep step: over
// 8192 terms that was measured as a relative error of 6e-6.  A tile is
// therefore summed in segments (MxGradParams::seg), and the draining warps
// add the segments in registers, rounding to nearest; the two accumulators in
// tensor memory let that overlap the next segment.
#include "mx.cuh"

namespace dgemm {
namespace {

constexpr int BK = kMxGradBK;
constexpr int kThreads = 640;
constexpr int kConvWarp = 4, kConvGroup = 4;              // two groups of 4 warps
constexpr int kEpiWarp = 12, kEpiWarps = 8;
// Registers per thread: 96 at launch; after the split 128 threads of loads
// and MMAs, 256 of conversion, 256 of draining (128 sums and 16 loaded
// values each): 32 + 2 * 56 + 2 * 168 = 5 * 96.
constexpr int kRegsLaunch = 96, kRegsIssue = 32, kRegsConv = 56, kRegsEpi = 168;
static_assert(kRegsIssue + 2 * kRegsConv + 2 * kRegsEpi <= 5 * kRegsLaunch, "register split");

// A stage is two halves of 64 of K, each with its part of both operands as
// 64-wide, 128-byte swizzled blocks; one barrier round trip of the MMA
// issuer covers eight MMAs (with stages of 64 it spent as long on its
// barriers as on the MMAs: 121 against 88 us at 4096^3).
constexpr int kHalves = BK / 64;
constexpr uint32_t kBlock = 64 * 64 * 2;                  // 64 wide, 64 deep: 8 KB
constexpr uint32_t kConvHalf = 2 * kBlock;                // 128 columns of B
constexpr uint32_t kAHalf = 2 * kBlock;                   // 128 rows of C
constexpr uint32_t kConvBytes = kHalves * kConvHalf;
constexpr uint32_t kABytes = kHalves * kAHalf;
constexpr uint32_t kStage = kConvBytes + kABytes;         // 64 KB
constexpr int S = 3;
constexpr uint32_t kTmemCols = 512;                       // two accumulators
static_assert(BK == kMxTileRows, "a stage needs one tile of scales per CTA");

template <int kFmt>
struct Layout {
  static constexpr uint32_t kRawRow = kFmt == GEMM_MXFP4 ? 64 : 128;   // 128 codes
  static constexpr uint32_t kRaw = kRawRow * BK;
  static constexpr uint32_t kRawStage = kRaw + kMxTileBytes;
  // (Even: a slot's stages all fall to one group of converting warps, which
  // therefore never waits for a phase whose predecessor it has not seen.)
  static constexpr int kRawStages = 2;
  static_assert(kRawStages % 2 == 0, "one group per slot");
  static constexpr uint32_t kSmem = S * kStage + kRawStages * kRawStage + 1024 + 512;
  static_assert(kSmem <= 232448, "shared memory");
};

template <int R>
struct alignas(8) Barriers {
  uint64_t full[S];       // even CTA: op(A) of both CTAs loaded, both conversions done
  uint64_t empty[S];      // the MMAs on stage s are done
  uint64_t raw_full[R];   // codes and scales of this CTA loaded
  uint64_t raw_empty[R];  // and read by the converting warps
  uint64_t acc_full[2];
  uint64_t acc_empty[2];  // even CTA
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

// ------------------------------------------------------------ conversion

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Byte permutation; a selector digit with its top bit set gives the sign of
// the byte that it selects, eight times.
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
  return r;
}
__device__ __forceinline__ uint32_t twice(uint32_t h) { return h | (h << 16); }

// FP16 bits of 2^e, e in [-24, 15].
__device__ __forceinline__ uint32_t f16_pow2(int e) {
  return e >= -14 ? (uint32_t)(e + 15) << 10 : 1u << (e + 24);
}

// A block's scale as multipliers of its values.  BF16: one, exact (2^-127 is
// a subnormal).  s * 0x00800080 puts s into both exponent fields; bit 6 of the
// fraction makes 2^-127 of s = 0 and NaN of s = 255.
// FP16: two powers of two whose product is the scale.  The first is at least
// 2^-14, so a value times it is exact (both formats' steps are 2^-6 or more)
// and only the second product rounds; the exponents below -39 that the clamp
// changes give zero either way, those above 30 infinity.
template <typename T>
struct Scale {
  uint32_t a, b;
  __device__ __forceinline__ explicit Scale(unsigned s) {
    if constexpr (__is_same(T, __nv_bfloat16)) {
      a = s * 0x00800080u;
      if (((s + 1u) & 0xFEu) == 0u) a |= 0x00400040u;
      b = 0;
    } else {
      const int e = (int)s - 127;
      const int e1 = min(max(e, -14), 15);
      const int e2 = min(max(e - e1, -25), 15);
      a = twice(s == 255u ? 0x7E00u : f16_pow2(e1));
      b = twice(e2 < -24 ? 0u : f16_pow2(e2));
    }
  }
  __device__ __forceinline__ uint32_t times(uint32_t v) const {
    if constexpr (__is_same(T, __nv_bfloat16)) return mul_bf16x2(v, a);
    return mul_f16x2(mul_f16x2(v, a), b);
  }
};

// Eight E2M1 codes as four pairs of 16-bit values, scaled.
template <typename T>
__device__ __forceinline__ uint4 convert_e2m1x8(uint32_t w, const Scale<T>& sc) {
  uint32_t r[4];
  if constexpr (__is_same(T, __nv_bfloat16)) {
    // prmt looks up four magnitudes 2 |x| = 0, 1, 2, 3, 4, 6, 8, 12 as bytes
    // and gives 0 where the selector's (the code's) top bit is set: with the
    // codes, and with their signs flipped, the positive and the negative
    // ones.  0xC0 + 2 x is the low byte of 96 + x in BF16 (high byte 0x42).
    const uint32_t flipped = w ^ 0x88888888u;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t pos = prmt(0x03020100u, 0x0C080604u, h == 0 ? w : w >> 16);
      const uint32_t neg = prmt(0x03020100u, 0x0C080604u, h == 0 ? flipped : flipped >> 16);
      const uint32_t sum = 0xC0C0C0C0u + pos - neg;   // (no byte carries)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        r[2 * h + j] = sc.times(
            sub_bf16x2(prmt(sum, 0x42424242u, j == 0 ? 0x4140 : 0x4342), 0x42C042C0u));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t h;
      asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
          "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
          "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
          : "=r"(h)
          : "r"(w >> (8 * j)));
      r[j] = sc.times(h);
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// Four MXINT8 codes as two pairs of 16-bit values, scaled.
template <typename T>
__device__ __forceinline__ uint2 convert_int8x4(uint32_t w, const Scale<T>& sc) {
  uint32_t r[2];
  if constexpr (__is_same(T, __nv_bfloat16)) {
    // A code c = low7 - 128 sign.  0x4000 + low7 is 2 + low7 / 64 in BF16 and
    // 0x4000 + (c & 0x80) is 2 (1 + sign): their difference is c / 64, exactly.
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t p = __byte_perm(w, 0x40404040u, j == 0 ? 0x4140 : 0x4342);
      r[j] = sc.times(sub_bf16x2(p & 0x407F407Fu, p & 0x40804080u));
    }
  } else {
    // 0x4C00 + u is 16 + u / 64 in FP16; u = c + 128.
    const uint32_t u = w ^ 0x80808080u;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t p = __byte_perm(u, 0x4C4C4C4Cu, j == 0 ? 0x4140 : 0x4342);
      r[j] = sc.times(sub_f16x2(p, 0x4C804C80u));
    }
  }
  return make_uint2(r[0], r[1]);
}

// ------------------------------------------------------------ kernel

template <int kFmt, typename T, typename TC, bool kAT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    mx_grad_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const MxGradParams p) {
  using L = Layout<kFmt>;
  constexpr int R = L::kRawStages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* const base = align_smem_1024(smem_raw);
  unsigned char* const sraw = base + S * kStage;
  auto* bars = reinterpret_cast<Barriers<R>*>(sraw + R * L::kRawStage);
  static_assert(sizeof(Barriers<R>) <= 512, "barrier block must fit its reserved space");
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();   // 0: issues the MMAs
  const int npairs = gridDim.x >> 1;
  const int nk = (p.K + BK - 1) / BK;
  const MxSchedule& sc = p.sched;
  constexpr uint32_t kAb = __is_same(T, __half) ? 0u : 1u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&bars->full[s]), 1 + 2 * kConvGroup);
      mbar_init(smem_u32(&bars->empty[s]), 1);
    }
    for (int r = 0; r < R; ++r) {
      mbar_init(smem_u32(&bars->raw_full[r]), 1);
      mbar_init(smem_u32(&bars->raw_empty[r]), kConvGroup);
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
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) tmem_alloc_pair(smem_u32(&bars->tmem_base), kTmemCols);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = bars->tmem_base;
  wait_prior_grids();
  allow_dependent_grids();

  uint32_t issued = 0;
  if (warp < kConvWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 0 && elect_one()) {
      // ---------------------------------------------- op(A) (both CTAs)
      RingPos<S> pos;
      uint32_t it = 0;
      bool ok = true;
      for (int u = blockIdx.x >> 1; u < sc.units && ok; u += npairs) {
        const MxUnit w = mx_unit(u, sc, nk);
        if (w.row0 >= p.M) continue;
        const int boxes = w.rows / 128;               // of 64 rows of C, per CTA
        const int row = w.row0 + (int)rank * (w.rows / 2);
        for (int kt = w.kb; kt < w.ke; ++kt, ++it, pos.next()) {
          const uint32_t s = pos.slot;
          ok = role_wait(smem_u32(&bars->empty[s]), pos.parity ^ 1u, p.fault, p.timeout_ns,
                         &bars->abort, kFaultTcProducerWait, true);
          if (!ok) break;
          const uint32_t sa = smem_u32(base + s * kStage) + kConvBytes;
          const uint32_t fb = mapa_shared(smem_u32(&bars->full[s]), 0);
          if (rank == 0)
            mbar_arrive_expect_tx(smem_u32(&bars->full[s]),
                                  2u * kHalves * (uint32_t)boxes * kBlock);
          for (int h = 0; h < kHalves; ++h) {
            const int k = kt * BK + h * 64;
            for (int j = 0; j < boxes; ++j) {
              const uint32_t dst = sa + h * kAHalf + j * kBlock;
              if constexpr (kAT)   // stored K x M: rows of C contiguous
                tma_load_2d_pair(dst, &tmA, fb, row + j * 64, k);
              else
                tma_load_2d_pair(dst, &tmA, fb, k, row + j * 64);
            }
          }
          issued = it + 1;
        }
      }
    } else if (warp == 2 && elect_one()) {
      // ---------------------------------------------- codes and scales (both CTAs)
      const int ktiles = mx_scale_tiles(p.N);
      RingPos<R> pos;
      uint32_t it = 0;
      bool ok = true;
      for (int u = blockIdx.x >> 1; u < sc.units && ok; u += npairs) {
        const MxUnit w = mx_unit(u, sc, nk);
        if (w.row0 >= p.M) continue;
        const int ct = w.tn * 2 + (int)rank;          // this CTA's 128 columns
        const uint32_t sbytes = ct < ktiles ? (uint32_t)kMxTileBytes : 0u;
        for (int kt = w.kb; kt < w.ke; ++kt, ++it, pos.next()) {
          const uint32_t r = pos.slot;
          ok = role_wait(smem_u32(&bars->raw_empty[r]), pos.parity ^ 1u, p.fault, p.timeout_ns,
                         &bars->abort, kFaultTcProducerWait, true);
          if (!ok) break;
          const uint32_t raw = smem_u32(sraw + r * L::kRawStage);
          const uint32_t rb = smem_u32(&bars->raw_full[r]);
          mbar_arrive_expect_tx(rb, L::kRaw + sbytes);
          tma_load_2d(raw, &tmB, rb, ct * (int)L::kRawRow, kt * BK);
          if (sbytes != 0)
            bulk_load(raw + L::kRaw,
                      p.sb + ((long long)kt * ktiles + ct) * kMxTileBytes, sbytes, rb);
          issued = it + 1;
        }
      }
    } else if (warp == 1 && rank == 0 && elect_one()) {
      // ---------------------------------------------- MMA issuer (even CTA)
      // The barrier of the next stage is tried before this stage's MMAs are
      // issued: a try takes over 100 cycles to answer.
      RingPos<S> pos;
      bool ready = false;
      uint32_t seg = 0;
      bool ok = true;
      for (int u = blockIdx.x >> 1; u < sc.units && ok; u += npairs) {
        const MxUnit w = mx_unit(u, sc, nk);
        if (w.row0 >= p.M) continue;
        const uint32_t idesc = instr_desc(kAb, 256, (uint32_t)w.rows, 1u, kAT ? 1u : 0u);
        for (int k0 = w.kb; k0 < w.ke && ok; k0 += p.seg, ++seg) {
          const int k1 = min(k0 + p.seg, w.ke);
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
            // MN-major tiles step by 16 rows of 128 bytes per 16 of K, K-major
            // ones by 32 bytes.
            const uint32_t blo = desc_lo(st, kBlock);
            const uint32_t alo = desc_lo(st + kConvBytes, kAT ? kBlock : 16);
#pragma unroll
            for (int k = 0; k < BK / 16; ++k)
              mma_f16_pair_lo(tmem_base + b * 256,
                              blo + (((k >> 2) * kConvHalf + (k & 3) * 2048) >> 4),
                              alo + (((k >> 2) * kAHalf + (k & 3) * (kAT ? 2048 : 32)) >> 4),
                              idesc, (kt > k0 || k > 0) ? 1u : 0u);
            mma_commit_pair_multicast(freed, 0x3);
          }
          if (!ok) break;
          mma_commit_pair_multicast(smem_u32(&bars->acc_full[b]), 0x3);
        }
      }
    }
    __syncwarp();
  } else if (warp < kEpiWarp) {
    // ------------------------------------------------ conversion of B (both CTAs)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConv));
    // The two groups of 4 warps take turns at the stages, so that one's waits
    // and fences pass while the other converts: half a stage each, in step,
    // left the ALUs idle for half of the time.
    // Lane l of warp v of its group takes the 16 columns 16 (l % 4) of the
    // 64-column block (l / 8) % 2, rows 4 v + (l / 4) % 2 + 2 (l / 16) + 16 i.
    // Eight lanes so store even chunks of one row and of the next, odd one,
    // whose swizzle swaps even and odd: no bank conflicts.
    const int group = (warp - kConvWarp) / kConvGroup;
    const int v = (warp - kConvWarp) % kConvGroup;
    const int unit = lane & 3, blk = (lane >> 3) & 1;
    const int row0 = 4 * v + ((lane >> 2) & 1) + 2 * (lane >> 4);
    const int column = blk * 64 + unit * 16;
    uint32_t first = 0;      // ring index of the unit's first stage
    bool ok = true;
    for (int u = blockIdx.x >> 1; u < sc.units && ok; u += npairs) {
      const MxUnit w = mx_unit(u, sc, nk);
      if (w.row0 >= p.M) continue;
      for (int kt = w.kb + (int)((group ^ first) & 1u); kt < w.ke; kt += 2) {
        const uint32_t it = first + (uint32_t)(kt - w.kb);
        const uint32_t r = it % R, s = it % S;
        // (Both tries are on their way at once.)
        const bool loaded = mbar_try_wait(smem_u32(&bars->raw_full[r]), (it / R) & 1u);
        const bool freed = mbar_try_wait(smem_u32(&bars->empty[s]), ((it / S) & 1u) ^ 1u);
        ok = role_wait_lanes(smem_u32(&bars->raw_full[r]), (it / R) & 1u, p.fault, p.timeout_ns,
                             &bars->abort, kFaultTcProducerWait, loaded);
        if (!ok) break;
#pragma unroll
        for (int half = 0; half < kHalves; ++half) {
          const unsigned char* raw = sraw + r * L::kRawStage + half * 64 * L::kRawRow;
          const unsigned char* scales =
              sraw + r * L::kRawStage + L::kRaw + half * 2 * 4 + (column >> 5);
          const int rows_left = p.K - kt * BK - half * 64;
          // All loads before the first store, which the compiler could not
          // move a load across.
          uint32_t c[4][kFmt == GEMM_MXFP4 ? 2 : 4];
          unsigned sb[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = row0 + 16 * i;
            if constexpr (kFmt == GEMM_MXFP4) {
              const uint2 x = *reinterpret_cast<const uint2*>(raw + row * L::kRawRow + column / 2);
              c[i][0] = x.x, c[i][1] = x.y;
            } else {
              const uint4 x = *reinterpret_cast<const uint4*>(raw + row * L::kRawRow + column);
              c[i][0] = x.x, c[i][1] = x.y, c[i][2] = x.z, c[i][3] = x.w;
            }
            sb[i] = scales[(row & 31) * 16 + (row >> 5) * 4];
            // Rows past K: zero codes, and any finite scale.
            if (row >= rows_left) sb[i] = 0;
          }
          if (half == 0)
            ok = role_wait_lanes(smem_u32(&bars->empty[s]), ((it / S) & 1u) ^ 1u, p.fault,
                                 p.timeout_ns, &bars->abort, kFaultTcProducerWait, freed);
          if (!ok) break;
          if (half == kHalves - 1) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->raw_empty[r]));
          }
          unsigned char* st = base + s * kStage + half * kConvHalf + blk * kBlock;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = row0 + 16 * i;
            const Scale<T> f(sb[i]);
            uint4 lo, hi;
            if constexpr (kFmt == GEMM_MXFP4) {
              lo = convert_e2m1x8<T>(c[i][0], f);
              hi = convert_e2m1x8<T>(c[i][1], f);
            } else {
              const uint2 a = convert_int8x4<T>(c[i][0], f), b = convert_int8x4<T>(c[i][1], f);
              const uint2 d = convert_int8x4<T>(c[i][2], f), e = convert_int8x4<T>(c[i][3], f);
              lo = make_uint4(a.x, a.y, b.x, b.y);
              hi = make_uint4(d.x, d.y, e.x, e.y);
            }
            unsigned char* dst = st + row * 128;
            *reinterpret_cast<uint4*>(dst + (((2 * unit) ^ (row & 7)) << 4)) = lo;
            *reinterpret_cast<uint4*>(dst + (((2 * unit + 1) ^ (row & 7)) << 4)) = hi;
          }
        }
        if (!ok) break;
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_any_cta(mapa_shared(smem_u32(&bars->full[s]), 0));
      }
      first += (uint32_t)(w.ke - w.kb);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ epilogue (both CTAs)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    // Warp: TMEM lanes 32 q .. 32 q + 31 (columns of C), half of the rows.
    const int q = warp & 3;
    const int half = (warp - kEpiWarp) >> 2;
    const bool pairs = (reinterpret_cast<uintptr_t>(p.C) & 3u) == 0 && ((p.ldc | p.N) & 1) == 0;
    uint32_t seg = 0;
    bool ok = true;
    for (int u = blockIdx.x >> 1; u < sc.units && ok; u += npairs) {
      const MxUnit w = mx_unit(u, sc, nk);
      if (w.row0 >= p.M) continue;
      const int chunks = w.rows / 64;      // of 32 rows, this warp's share
      const int first = half * (w.rows / 2);
      float acc[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) acc[j] = 0.f;
      for (int k0 = w.kb; k0 < w.ke; k0 += p.seg, ++seg) {
        const uint32_t b = seg & 1;
        ok = role_wait_lanes(smem_u32(&bars->acc_full[b]), (seg >> 1) & 1u, p.fault, p.timeout_ns,
                             &bars->abort, kFaultTcEpilogueWait, false, false);
        if (!ok) break;
        tc_fence_after();
        const uint32_t t = tmem_base + ((uint32_t)(q * 32) << 16) + b * 256 + first;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (c < 2 * chunks) {
            uint32_t r[16];
            tmem_ld16(t + c * 16, r);
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[c * 16 + j] += __uint_as_float(r[j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_any_cta(mapa_shared(smem_u32(&bars->acc_empty[b]), 0));
      }
      if (!ok) break;
      const int col = w.tn * 256 + (int)rank * 128 + q * 32 + lane;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (c < chunks) {
          const int row = w.row0 + first + c * 32;
          const float* v = acc + c * 32;
          if (sc.slices == 1)
            store_piece<TC>(v, static_cast<TC*>(p.C), p.ldc, p.M, p.N, row, col, pairs, p.alpha,
                            p.beta);
          else if (col < p.N)
            store_rows32<float>(v, p.ws + ((long long)w.slice * p.M + row) * p.ldw + col, p.ldw,
                                p.M - row, 1.f, 0.f);
        }
      }
    }
  }

  // ------------------------------------------------ teardown
  if (warp == 1 && rank == 0 && elect_one()) {
    // Every MMA of the pair has completed before TMEM is freed.
    mma_commit_pair_multicast(smem_u32(&bars->drain), 0x1);
    if (!mbar_wait_bounded(smem_u32(&bars->drain), 0, p.timeout_ns, nullptr))
      raise_fault(p.fault, kFaultDrainWait);
  }
  __syncthreads();
  if ((warp == 2 || (warp == 0 && rank == 0)) && elect_one() && bars->abort) {
    // Let the copies in flight land: those of codes on raw_full[], and those
    // of op(A), both CTAs', on the even one's full[], whose arrivals by
    // converting warps may be missing; the wait then gives up.
    const uint32_t n = warp == 2 ? R : S;
    const uint32_t first = issued > n ? issued - n : 0;
    for (uint32_t it = first; it < issued; ++it) {
      const uint64_t* bar = warp == 2 ? &bars->raw_full[it % R] : &bars->full[it % S];
      if (!mbar_wait_bounded(smem_u32(bar), (it / n) & 1u, p.timeout_ns, nullptr)) {
        raise_fault(p.fault, kFaultDrainWait);
        break;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // neither CTA leaves while the pair may still touch its memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

template <int kFmt, typename T, typename TC, bool kAT>
cudaError_t launch_typed(const MxGradParams& p, const CUtensorMap* tmA, const CUtensorMap* tmB,
                         int pairs, cudaStream_t stream) {
  auto kernel = mx_grad_kernel<kFmt, T, TC, kAT>;
  // The register split needs kRegsLaunch registers a thread at launch: with
  // fewer, its setmaxnreg.inc would wait for ever.
  static const bool fits = [&] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, kernel) == cudaSuccess && a.numRegs == kRegsLaunch;
  }();
  if (!fits) return cudaErrorInvalidConfiguration;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = mx_allow_smem(kernel, Layout<kFmt>::kSmem, &done);
  if (e != cudaSuccess) return e;
  return launch_gemm_kernel(kernel, dim3(2 * pairs), dim3(kThreads), Layout<kFmt>::kSmem, stream,
                            *tmA, *tmB, p);
}

template <int kFmt, typename T>
cudaError_t launch_fmt(const MxGradParams& p, const CUtensorMap* a, const CUtensorMap* b,
                       int pairs, cudaStream_t s) {
  if (p.dtype_c == 0)
    return p.op_a ? launch_typed<kFmt, T, float, true>(p, a, b, pairs, s)
                  : launch_typed<kFmt, T, float, false>(p, a, b, pairs, s);
  return p.op_a ? launch_typed<kFmt, T, T, true>(p, a, b, pairs, s)
                : launch_typed<kFmt, T, T, false>(p, a, b, pairs, s);
}

}  // namespace

cudaError_t launch_mx_grad(const MxGradParams& p, const CUtensorMap* a, const CUtensorMap* b,
                           int pairs, cudaStream_t s) {
  if (p.dtype == 1)
    return p.fmt == GEMM_MXFP4 ? launch_fmt<GEMM_MXFP4, __half>(p, a, b, pairs, s)
                               : launch_fmt<GEMM_MXINT8, __half>(p, a, b, pairs, s);
  return p.fmt == GEMM_MXFP4 ? launch_fmt<GEMM_MXFP4, __nv_bfloat16>(p, a, b, pairs, s)
                             : launch_fmt<GEMM_MXINT8, __nv_bfloat16>(p, a, b, pairs, s);
}

}  // namespace dgemm
