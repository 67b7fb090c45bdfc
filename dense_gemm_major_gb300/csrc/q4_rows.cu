// Products with 4-bit weights and group scales on tcgen05, of tiles of up to 128 rows:
// Y = X . W^T, the weights rounded to X's type on the way.
//
// Bound by reading the codes and by the instructions that make 16-bit values of them
// (for eight codes 8 or 9 of the integer and 8 of the FMA pipe, each at half rate), which
// do not depend on the number of rows; so W is the MMA's M side (128 rows per CTA), X
// its N side (16 to 128).  The values go to tensor memory, from where the MMA reads its
// A: through shared memory they would be written and read at four times the codes'
// bytes, which is what bounded a first version (8192 x 8192, 16 rows: 19.8 us).  A
// thread has a row of W, as a lane of tensor memory has.
//
// The rounding of the weights is a choice for speed.  Integers whose sums are scaled group by
// group, as in q4_few.cu, would be exact, but the sums would leave tensor memory once for each
// 32 to 128 terms, a value for each of up to 128 rows and lane, rather than once.  Error of the
// result against 64 bits, of its norm: 2.2e-3 in BF16, for 1.66e-3 of the result's rounding alone.
//
// Few units: so that W's bytes travel to all SMs at once, the CTAs of a cluster share a
// tile's K; they add their FP32 partial tiles through distributed shared memory in rank order,
// so results are reproducible and there is no workspace.  Many (kLoop): a CTA goes from unit
// to unit, with two accumulators in turn, so that loads and conversions do not stop between
// them (a unit for each CTA of a larger grid: 512 rows of 64 experts, 2048 x 2048, 66.9 -> 42.6
// us, 2048 of 32 49.8 -> 31.2, 512 x 8192 x 8192 57.1 -> 48.7).
//
// Measured in a graph on changing weights, BF16, groups of 128: 40 x 8192 x 8192 14.2 us
// (2.5 TB/s of codes and scales), 33 x 4096 x 4096 7.5, 128 x 4096 x 4096 9.8; 1024 x 4096 x
// 4096 29.1, 2048 x 8192 x 8192 166 (1.66 PFLOP/s).  What bounds 40 rows: the turns of the
// converting warps, some 4 us before and after them (without the conversions 12 us), and 24 of
// the 152 SMs, which 64 tiles leave idle.  768 x 8192 x 8192: 72.9, without the
// conversions 63, with one MMA of eight 62.
//
// Roles (640 threads): warp 0 loads the codes (TMA) into a ring of their own, warp 1
// issues the MMAs, warp 2 loads X, warps 4-19 convert: four groups of 4 warps take turns
// at 128-deep stages, so that one's waits pass while the others convert.  Each group drains
// some rows of the accumulators.
#include "q4.cuh"

namespace dgemm {
namespace {

constexpr int BN = kQ4RowsTileN, BK = kQ4RowsBK;
constexpr int kThreads = 640;
constexpr int kConvWarp = 4, kGroups = 4, kGroupWarps = 4;
// A slot of codes is two stages deep: TMA then copies 128 bytes of each row.  (With that
// and four groups of converting warps, for two groups of 8 and slots of one stage, 17.3 ->
// 15.8 us at 8192 x 8192, 16 rows.)
constexpr uint32_t kRawBytes = BN * BK;                     // 16 KB
constexpr uint32_t kACols = BK / 2;                         // of tensor memory, a stage of W
// Units from the one that a warp drains next to the one of its next stage: of two stages or
// more, so that a turn is two units ahead of the last, and the next one four.
constexpr uint32_t kEntered = 8;

// MT: rows of X that the MMA computes.  kLoop: a CTA goes from unit to unit; else it has a
// share of K of only one.
template <int MT, bool kLoop>
struct Layout {
  static constexpr uint32_t kXBlock = MT * 128;             // 64 k of X
  static constexpr uint32_t kStage = 2 * kXBlock;
  // A group may only wait for a phase whose predecessor is known to be over.  Slots of
  // codes: their number is even, so that each is read by the same two groups every time.
  // Stages: the MMAs free them in order, and a group has seen the one freed that it
  // waited for kGroups stages ago, so that there need to be that many.
  static constexpr int S = MT <= 64 ? 6 : 4, R = kLoop && MT > 64 ? 4 : 6;
  static_assert(S >= kGroups && R % 2 == 0, "phases");
  static constexpr uint32_t kTable =
      kLoop ? (sizeof(Q4Tables) + 15) / 16 * 16 + kGroups * kGroupWarps * kEntered * 16 : 0;
  // All of an SM's (s_unit is beside it), so that no CTA of another cluster with tensor
  // memory is: two clusters could each hold on one SM what the other waits for on another.
  static constexpr uint32_t kSmem = 232448 - 1024;
  static_assert(S * kStage + R * kRawBytes + kTable + 512 + 1024 <= kSmem, "shared memory");
  static_assert(MT * BN * 4 <= S * kStage + R * kRawBytes, "partial tiles reuse the rings");
  // Tensor memory: the accumulator (two, in turn), then W's stages.
  static constexpr uint32_t kAccCols = MT < 32 ? 32 : MT;
  static constexpr uint32_t kACol = kLoop ? 2 * kAccCols : kAccCols;
  static_assert(kACol + S * kACols <= 512, "tensor memory");
  // Warps that drain an accumulator: each group takes every fourth 16 rows of X.
  static constexpr int kDrainWarps = kGroupWarps * (MT / 16 < kGroups ? MT / 16 : kGroups);
};

template <int S, int R>
struct alignas(8) Barriers {
  uint64_t full[S];       // X loaded, W converted
  uint64_t empty[S];
  uint64_t raw_full[R];
  uint64_t raw_empty[R];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

// 16-deep step with A in tensor memory: 128 lanes by 8 columns of pairs; B as in
// mma_f16_pair_lo.
__device__ __forceinline__ void mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint32_t blo,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(blo), "r"(kDescHi128B), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Eight codes as four pairs of weights over kQ4Value, in the order of their columns; z:
// the zero, s: the scale, twice (see zero_term()).  FP16: a code in the low mantissa bits of
// 1024 is that plus the code.  BF16: the integer n in a number's low eight bits is n
// 2^-133, so that 2^127 and, four bits further up, 2^123 make both codes of a byte q / 64.
template <typename T>
__device__ __forceinline__ void weights8(uint32_t w, uint32_t z, uint32_t s, uint32_t* v) {
  const uint32_t h = w >> 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (__is_same(T, __half)) {
      // Byte j of the low and of the high halves; the other bytes are masked away.
      const uint32_t x = __byte_perm(w, h, (j + 4) * 0x1100 + j * 0x11);
      v[j] = mul_x2<T>(fma_x2<T>(and_or(x, 0x000F000Fu, 0x64006400u), 0x3C003C00u, z), s);
    } else {
      const uint32_t x = __byte_perm(w, w, j * 0x1111) & 0x00F0000Fu;
      v[j] = mul_x2<T>(fma_x2<T>(x, 0x7D007F00u, z), s);
    }
  }
}
// -(1024 + zero) in FP16, -zero / 64 in BF16, twice.
template <typename T>
__device__ __forceinline__ uint32_t zero_term(uint32_t zero) {
  if constexpr (__is_same(T, __half)) return 0xE400E400u + zero * 0x00010001u;
  const float v = (float)zero * -0x1p-6f;
  return pack2<T>(v, v);
}

// kRun: columns that have one scale (32, 64, or a stage's 128).
template <typename T, int MT, int kRun, bool kLoop>
__global__ void __launch_bounds__(kThreads, 1)
    q4_rows_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmX,
                   const Q4FewParams p) {
  using L = Layout<MT, kLoop>;
  constexpr int S = L::S, R = L::R;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* const base = align_smem_1024(smem_raw);
  unsigned char* const raw_base = base + S * L::kStage;
  auto* bars = reinterpret_cast<Barriers<S, R>*>(raw_base + R * kRawBytes);
  static_assert(sizeof(Barriers<S, R>) <= 512, "barrier block must fit its reserved space");
  // (kLoop:) each converting warp's units since the one it drains next, the tables.
  int4* const entered = reinterpret_cast<int4*>(raw_base + R * kRawBytes + 512);
  Q4Tables& tables = *reinterpret_cast<Q4Tables*>(entered + kGroups * kGroupWarps * kEntered);
  __shared__ Q4Unit s_unit;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = !kLoop && p.split > 1 ? (int)cluster_ctarank() : 0;
  // This CTA's k-tiles of a unit: from kb on (even), of which there are `stages`.  (In a loop
  // they are even too, the last one all zeros if need be: every unit begins with a slot.)
  const int nk = (p.K + BK - 1) / BK, nk2 = (nk + 1) / 2;
  const int kb = kLoop ? 0 : 2 * (int)((long long)rank * nk2 / p.split);
  const int stages =
      kLoop ? 2 * nk2 : min(2 * (int)((long long)(rank + 1) * nk2 / p.split), nk) - kb;
  // (kLoop: from unit to unit; else the one that the grid gives.)
  const Q4Walk walk0(p.N, BN, blockIdx.x / (unsigned)p.split, gridDim.x);
  constexpr uint32_t kAb = __is_same(T, __half) ? 0u : 1u;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&bars->full[s]), 1 + kGroupWarps);
      mbar_init(smem_u32(&bars->empty[s]), 1);
    }
    for (int r = 0; r < R; ++r) {
      mbar_init(smem_u32(&bars->raw_full[r]), 1);
      mbar_init(smem_u32(&bars->raw_empty[r]), 2 * kGroupWarps);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&bars->acc_full[b]), 1);
      mbar_init(smem_u32(&bars->acc_empty[b]), L::kDrainWarps);
    }
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) tmem_alloc(smem_u32(&bars->tmem_base), 512);
  wait_prior_grids();
  allow_dependent_grids();
  if (warp == 2) {
    Q4Unit w;
    if constexpr (kLoop) {
      w = q4_tables(p, tables, walk0.slot);
    } else {
      const Q4Rows r = q4_rows_of_slot((int)blockIdx.y, p);
      w = Q4Unit{r.expert, r.lo, r.hi, 0, r.expert >= 0};
    }
    w.n0 = walk0.n * BN;
    if (lane == 0) s_unit = w;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = bars->tmem_base;
  const Q4Unit unit0 = s_unit;
  if (!unit0.real) {   // (the same in all of a cluster)
    if (warp == 1) tmem_dealloc(tmem_base, 512);
    return;
  }

  uint32_t issued = 0;
  if (warp == 0) {
    if (elect_one()) {
      // ---------------------------------------------- codes
      RingPos<R> pos;
      bool ok = true;
      Q4Unit unit = unit0;
      for (Q4Walk walk = walk0; ok && unit.real;) {
        for (int kt = kb; kt < kb + stages; kt += 2, pos.next()) {
          ok = role_wait(smem_u32(&bars->raw_empty[pos.slot]), pos.parity ^ 1u, p.fault,
                         p.timeout_ns, &bars->abort, kFaultTcProducerWait, true);
          if (!ok) break;
          const uint32_t full = smem_u32(&bars->raw_full[pos.slot]);
          mbar_arrive_expect_tx(full, kRawBytes);
          tma_load_3d(smem_u32(raw_base + pos.slot * kRawBytes), &tmQ, full, kt * (BK / 2),
                      unit.n0, unit.expert);
          ++issued;
        }
        if (!kLoop) break;
        walk.next();
        unit = q4_unit(p, tables, walk, BN);
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    if (elect_one()) {
      // ---------------------------------------------- X
      RingPos<S> pos;
      bool ok = true;
      Q4Unit unit = unit0;
      for (Q4Walk walk = walk0; ok && unit.real;) {
        for (int kt = kb; kt < kb + stages; ++kt, pos.next()) {
          ok = role_wait(smem_u32(&bars->empty[pos.slot]), pos.parity ^ 1u, p.fault, p.timeout_ns,
                         &bars->abort, kFaultTcProducerWait, true);
          if (!ok) break;
          const uint32_t full = smem_u32(&bars->full[pos.slot]);
          const uint32_t to = smem_u32(base + pos.slot * L::kStage);
          mbar_arrive_expect_tx(full, 2 * L::kXBlock);
          tma_load_2d(to, &tmX, full, kt * BK, unit.lo);
          tma_load_2d(to + L::kXBlock, &tmX, full, kt * BK + 64, unit.lo);
          ++issued;
        }
        if (!kLoop) break;
        walk.next();
        unit = q4_unit(p, tables, walk, BN);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      // ---------------------------------------------- MMA issuer
      // (The barrier of the next stage is tried before this stage's MMAs are issued: a
      // try takes over 100 cycles to answer.)
      RingPos<S> pos;
      bool ok = true, ready = false;
      uint32_t n = 0;           // units
      Q4Walk walk = walk0;
      for (bool real = true; ok && real; ++n) {
        const uint32_t b = n & 1;
        if (kLoop) {
          ok = role_wait(smem_u32(&bars->acc_empty[b]), ((n >> 1) & 1u) ^ 1u, p.fault,
                         p.timeout_ns, &bars->abort, kFaultTcMmaWait, true);
          if (!ok) break;
          tc_fence_after();
        }
        for (int i = 0; i < stages; ++i) {
          const uint32_t slot = pos.slot;
          ok = ready || role_wait(smem_u32(&bars->full[slot]), pos.parity, p.fault, p.timeout_ns,
                                  &bars->abort, kFaultTcMmaWait, true);
          if (!ok) break;
          tc_fence_after();
          pos.next();
          ready = mbar_try_wait(smem_u32(&bars->full[pos.slot]), pos.parity);
          const uint32_t blo = desc_lo(smem_u32(base + slot * L::kStage), 16);
          const uint32_t a = tmem_base + L::kACol + slot * kACols;
#pragma unroll
          for (int k = 0; k < BK / 16; ++k)
            mma_f16_ta(tmem_base + b * L::kAccCols, a + k * 8,
                       blo + (((k >> 2) * L::kXBlock + (k & 3) * 32) >> 4),
                       instr_desc(kAb, BN, MT, 0, 0), (i > 0 || k > 0) ? 1u : 0u);
          mma_commit(smem_u32(&bars->empty[slot]));
        }
        if (ok) mma_commit(smem_u32(&bars->acc_full[b]));
        walk.next();
        real = kLoop && walk.slot < tables.slots;
      }
    }
    __syncwarp();
  } else if (warp >= kConvWarp) {
    // ------------------------------------------------ conversion
    // A thread of its group has a row.  (A warp reaches the lanes 32 (warp % 4) .. + 31.)
    constexpr int kRuns = BK / kRun;
    const int group = (warp - kConvWarp) / kGroupWarps;
    const int row = (warp & 3) * 32 + lane;
    // The scales and zeros of its runs, read a turn ahead and left as they come.
    const uint16_t* scales;
    const unsigned char* zeros;
    bool real;
    uint16_t sc[kRuns];
    unsigned char zr[kRuns];
    const int far_at = kGroups * BK / p.group, far_pos = kGroups * BK % p.group;
    int at, pos_in;
    // Its next stage: kt of the n-th unit (none beyond the last).
    Q4Walk walk = walk0;
    uint32_t n = 0;
    int kt = group, expert = 0;
    bool more;
    auto enter = [&](Q4Unit unit) {
      for (;;) {
        if constexpr (kLoop) {
          if (lane == 0 && unit.real)
            entered[(warp - kConvWarp) * kEntered + n % kEntered] =
                make_int4(unit.lo, unit.hi, unit.n0, 0);
        }
        expert = unit.expert;
        more = unit.real;
        if (!more || kt < stages) break;
        kt -= stages, ++n;
        if constexpr (kLoop) {
          walk.next();
          unit = q4_unit_by_warp(p, tables, walk, BN, expert);
        } else {
          unit.real = false;
        }
      }
      if (!more) return;
      const long long first_of_row =
          (long long)expert * q4_groups(p.K, p.group) * p.N + unit.n0 + row;
      scales = static_cast<const uint16_t*>(p.scales) + first_of_row;
      zeros = p.zeros != nullptr ? p.zeros + first_of_row : nullptr;
      real = unit.n0 + row < p.N;
      at = (kb + kt) * BK / p.group;
      pos_in = (kb + kt) * BK % p.group;
    };
    auto read_scales = [&] {
      int a = at, q = pos_in;
#pragma unroll
      for (int i = 0; i < kRuns; ++i) {
        const bool ok = real && more && (kb + kt) * BK + i * kRun < p.K;
        const long long to = (long long)a * p.N;
        sc[i] = ok ? scales[to] : (uint16_t)0;
        zr[i] = ok && zeros != nullptr ? zeros[to] : (unsigned char)8;
        if ((q += kRun) == p.group) q = 0, ++a;
      }
    };
    // 16-byte chunks in 128-byte rows are swizzled by the row; a stage has four.
    uint32_t from[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      from[i] = row * 128 + ((((group & 1) * 4 + i) ^ (row & 7)) << 4);
    const uint32_t lanes = tmem_base + ((uint32_t)((warp & 3) * 32) << 16);
    bool ok = true;
    // ------------------------------------------------ draining
    // Of the n-th unit, each group some rows.
    auto drain = [&](uint32_t n) {
      if (group * 16 >= MT) return;
      const uint32_t b = n & 1;
      const int4 unit = kLoop ? entered[(warp - kConvWarp) * kEntered + n % kEntered]
                              : make_int4(unit0.lo, unit0.hi, unit0.n0, 0);
      const int m_end = unit.y - unit.x;
      ok = role_wait_lanes(smem_u32(&bars->acc_full[b]), (n >> 1) & 1u, p.fault, p.timeout_ns,
                           &bars->abort, kFaultTcEpilogueWait);
      if (!ok) return;
      tc_fence_after();
#pragma unroll 1
      for (int c = group; c < MT / 16 && c * 16 < m_end; c += kGroups) {
        uint32_t r[16];
        tmem_ld16(lanes + b * L::kAccCols + c * 16, r);
        if constexpr (!kLoop) {
          // The partial tile, row-major, where the ring was.
          float* const part = reinterpret_cast<float*>(base) + c * 16 * BN + row;
#pragma unroll
          for (int j = 0; j < 16; ++j) part[j * BN] = __uint_as_float(r[j]);
        } else if (unit.z + row < p.N) {
          T* const y = static_cast<T*>(p.Y) + (long long)(unit.x + c * 16) * p.ldy + unit.z + row;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c * 16 + j < m_end)
              y[j * p.ldy] = from_f32_any<T>(__uint_as_float(r[j]) * kQ4Value<T>);
        }
      }
      if constexpr (kLoop) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->acc_empty[b]));
      }
    };
    uint32_t drained = 0, last = 0;      // (last: unit of the last turn's stage)
    enter(unit0);
    read_scales();
    for (uint32_t it = (uint32_t)group;; it += kGroups) {
      const bool now = more;
      const uint32_t turn = n;  // this stage's unit
      if (now) {
        const uint32_t r = (it / 2) % R, s = it % S;
        const uint32_t raw_parity = (it / 2 / R) & 1u, parity = ((it / S) & 1u) ^ 1u;
        // (Both tries are on their way at once.)
        const bool loaded = mbar_try_wait(smem_u32(&bars->raw_full[r]), raw_parity);
        const bool freed = mbar_try_wait(smem_u32(&bars->empty[s]), parity);
        uint32_t sv[kRuns], zv[kRuns];
#pragma unroll
        for (int i = 0; i < kRuns; ++i) {
          sv[i] = sc[i] * 0x00010001u;
          zv[i] = zero_term<T>(zr[i] & 15u);
        }
        const int terms = p.K - (kb + kt) * BK;     // from this stage on
        kt += kGroups;
        at += far_at;
        if ((pos_in += far_pos) >= p.group) pos_in -= p.group, ++at;
        if constexpr (kLoop) {
          if (kt >= stages) {
            kt -= stages, ++n;
            walk.next();
            enter(q4_unit_by_warp(p, tables, walk, BN, expert));
          }
        } else {
          more = kt < stages;
          n = more ? 0u : 1u;
        }
        read_scales();
        ok = role_wait_lanes(smem_u32(&bars->raw_full[r]), raw_parity, p.fault, p.timeout_ns,
                             &bars->abort, kFaultTcProducerWait, loaded);
        if (!ok) break;
        const uint32_t raw = smem_u32(raw_base) + r * kRawBytes;
        uint4 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = ld_shared_v4(raw + from[i]);
        if constexpr (__is_same(T, __half)) {
          // Past K, where X is zeros, codes less their zeros may overflow: there they
          // become their zeros.  (In BF16 they are below 1 before the scale.)
          if (terms < BK) {
            uint32_t* const words = reinterpret_cast<uint32_t*>(q);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint32_t none = (zv[i * 8 / kRun] & 15u) * 0x11111111u;
              const int left = terms - 8 * i;
              const uint32_t mask =
                  left >= 8 ? 0xFFFFFFFFu : (left > 0 ? (1u << 4 * left) - 1 : 0u);
              words[i] = (words[i] & mask) | (none & ~mask);
            }
          }
        }
        ok = role_wait_lanes(smem_u32(&bars->empty[s]), parity, p.fault, p.timeout_ns,
                             &bars->abort, kFaultTcProducerWait, freed);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a[32];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint4 x = q[2 * h + i];
            const int run = (2 * h + i) * 32 / kRun;
            const uint32_t sr = sv[run], zz = zv[run];
            weights8<T>(x.x, zz, sr, a + 16 * i);
            weights8<T>(x.y, zz, sr, a + 16 * i + 4);
            weights8<T>(x.z, zz, sr, a + 16 * i + 8);
            weights8<T>(x.w, zz, sr, a + 16 * i + 12);
          }
          tmem_st32(lanes + L::kACol + s * kACols + h * 32, a);
        }
        // (The proxy fence waits for the loads, before TMA refills the slot.)
        fence_proxy_async_smem();
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bars->full[s]));
          mbar_arrive(smem_u32(&bars->raw_empty[r]));
        }
      }
      // A unit is drained a turn after the next one's first, when its MMAs are done; but all
      // units before the last one are, whose accumulator the MMAs ahead may wait for: the
      // stage that this group's next turn waits for is of this turn's unit or before.
      const uint32_t over = !now ? n : max(last, turn == 0 ? 0u : turn - 1);
      last = turn;
      while (ok && drained < over) drain(drained++);
      if (!ok || !now) break;
    }
  }
  if constexpr (!kLoop) {
    // ------------------------------------------------ sum of the cluster's partial tiles
    cluster_sync_all();
    const Q4Unit rows = unit0;
    const int n0 = rows.n0;
    // This CTA adds up its part of the columns, four of a row per thread, all partial tiles'
    // values on their way at once.  (Only those that are stored are read: see
    // cluster_arrive_relaxed().)
    constexpr int kMaxSplit = 8;
    const int share = (BN / 4 + p.split - 1) / p.split;
    for (int i = threadIdx.x; i < share * (rows.hi - rows.lo); i += kThreads) {
      const int m = i / share;
      const int col = (rank * share + (i - m * share)) * 4;
      if (col >= BN || n0 + col >= p.N) continue;
      const uint32_t from = smem_u32(base) + (uint32_t)(m * BN + col) * 4u;
      float4 v[kMaxSplit];
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r)
        v[r] = r < p.split ? ld_cluster_v4(mapa_shared(from, (uint32_t)r))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
      float sum[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int r = 1; r < kMaxSplit; ++r) {
        sum[0] += v[r].x;
        sum[1] += v[r].y;
        sum[2] += v[r].z;
        sum[3] += v[r].w;
      }
      T* const y = static_cast<T*>(p.Y) + (long long)(rows.lo + m) * p.ldy + n0 + col;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n0 + col + j < p.N) y[j] = from_f32_any<T>(sum[j] * kQ4Value<T>);
    }
    // Nobody leaves while its sums may still be read.
    cluster_arrive_relaxed();
    cluster_wait();
  }

  // ------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if ((warp == 0 || warp == 2) && elect_one() && bars->abort) {
    // Let the copies in flight land; a stage of which conversions are missing makes
    // the wait give up.
    const uint32_t n = warp == 0 ? R : S;
    for (uint32_t i = issued > n ? issued - n : 0; i < issued; ++i) {
      const uint64_t* const bar = warp == 0 ? &bars->raw_full[i % R] : &bars->full[i % S];
      if (!mbar_wait_bounded(smem_u32(bar), (i / n) & 1u, p.timeout_ns, nullptr)) {
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
    tmem_dealloc(tmem_base, 512);
  }
}

template <typename T, int MT, int kRun, bool kLoop>
cudaError_t launch_kernel(const Q4FewParams& p, const CUtensorMap* tmQ, const CUtensorMap* tmX,
                          cudaStream_t stream) {
  using L = Layout<MT, kLoop>;
  auto kernel = q4_rows_kernel<T, MT, kRun, kLoop>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = mx_allow_smem(kernel, L::kSmem, &done);
  if (e != cudaSuccess) return e;
  const long long tiles = ((long long)p.N + BN - 1) / BN, units = tiles * p.slots;
  if (kLoop)
    return launch_gemm_kernel(kernel, dim3((unsigned)(units < p.max_ctas ? units : p.max_ctas)),
                              dim3(kThreads), L::kSmem, stream, *tmQ, *tmX, p);
  return launch_gemm_kernel_clusters((unsigned)p.split, kernel,
                                     dim3((unsigned)(tiles * p.split), (unsigned)p.slots),
                                     dim3(kThreads), L::kSmem, stream, *tmQ, *tmX, p);
}

template <typename T, int MT, int kRun>
cudaError_t launch_rows(const Q4FewParams& p, const CUtensorMap* q, const CUtensorMap* x,
                        cudaStream_t stream) {
  return p.split > 1 ? launch_kernel<T, MT, kRun, false>(p, q, x, stream)
                     : launch_kernel<T, MT, kRun, true>(p, q, x, stream);
}

template <typename T, int kRun>
cudaError_t launch_typed(const Q4FewParams& p, const CUtensorMap* q, const CUtensorMap* x,
                         cudaStream_t stream) {
  switch (p.tile_rows) {
    case 16: return launch_rows<T, 16, kRun>(p, q, x, stream);
    case 32: return launch_rows<T, 32, kRun>(p, q, x, stream);
    case 64: return launch_rows<T, 64, kRun>(p, q, x, stream);
    case 128: return launch_rows<T, 128, kRun>(p, q, x, stream);
  }
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch_run(const Q4FewParams& p, const CUtensorMap* q, const CUtensorMap* x,
                       cudaStream_t stream) {
  if (p.group % 128 == 0) return launch_typed<T, 128>(p, q, x, stream);
  return p.group % 64 == 0 ? launch_typed<T, 64>(p, q, x, stream)
                           : launch_typed<T, 32>(p, q, x, stream);
}

}  // namespace

int q4_rows_clusters(int split) {
  static std::atomic<int> known[9][64];
  return clusters_at_once(q4_rows_kernel<__half, 64, 128, false>, (unsigned)split, kThreads,
                          Layout<64, false>::kSmem, known[split]);
}

cudaError_t launch_q4_rows(int dtype, const Q4FewParams& p, const CUtensorMap* tmQ,
                           const CUtensorMap* tmX, cudaStream_t stream) {
  return dtype == 1 ? launch_run<__half>(p, tmQ, tmX, stream)
                    : launch_run<__nv_bfloat16>(p, tmQ, tmX, stream);
}

}  // namespace dgemm
