// Products of a few rows with 4-bit weights and group scales: Y = X . W^T,
// W[n][k] = s[n][k / group] (q[n][k] - z[n][k / group]).
//
// A CTA takes 64 rows of W and a share of K; its 8 warps are 2 groups of 32 rows x 4
// ranges of a stage's K, and multiply with mma.sync.m16n8k16: W's rows on the 16-wide
// side, X's on the 8-wide one.  The integers q - z are exact in 16 bits; each group's sum
// is kept apart in FP32 and scaled once, so that no product is rounded.  (On tcgen05, as
// in q4_rows.cu, a call takes 1 to 2 us longer up to 8 rows: tensor memory and its
// hand-overs, and a multiplication by the scale for every two weights.)
//
// Codes and X come by TMA into a ring.  The sum's order is free as long as both
// operands have it: a thread's word of eight codes is taken apart as the pairs (0,
// 4), (1, 5), (2, 6), (3, 7), a mask and a multiply-add each and one shift, and X's eight
// values are permuted the same way.  The four ranges of K and then the CTAs of the
// cluster are added in their order.
//
// Units of experts: a CTA goes from one to the next, whose first loads are under way at the
// end of each (a CTA for each unit: 64 rows of 64 experts, 2048 x 2048, 49.2 -> 37.6 us).
//
// Measured in a graph on changing weights, BF16, groups of 128: 1 x 4096 x 4096 5.2 us, 1 x
// 8192 x 8192 11.5 (3.0 TB/s of codes and scales; of 64: 12.4, of 32: 14.3), 32768 x 8192 35
// (4.0 TB/s).  Without the products 1 x 8192 x 8192 takes 9.  No unit is near its limit there
// (of the time: integer pipe 27 %, issue 31 %, DRAM 30 %).  What bounds it is latency: a warp
// waits for a stage, reads, converts and multiplies one after the other, with 16 such warps on
// an SM; and shares are uneven, 256 CTAs for 304 places leave 48 SMs with one.
#include "q4.cuh"

namespace dgemm {
namespace {

constexpr int kWarpsN = 2, kWarpsK = 4, kWarps = kWarpsN * kWarpsK;
constexpr int kThreads = 32 * (kWarps + 1);               // and one that loads
constexpr int kSliceK = kQ4BK / kWarpsK;                   // of a stage, per warp: 128
constexpr uint32_t kCodeBox = 128 * kQ4TileN;              // 256 codes of each row: 8 KB
constexpr int kCodeBoxes = kQ4BK / 256, kXBoxes = kQ4BK / 64;
static_assert(kWarpsN * 32 == kQ4TileN, "32 rows of W per warp");

// kTiles: 8-row tiles of X.  kExperts: a CTA goes from unit to unit, so that the next one's
// first loads are under way at the end of each; else it has only one.
template <int kTiles, bool kExperts>
struct Layout {
  static_assert(kTiles == 1 || !kExperts, "tiles of 8 rows of an expert");
  static constexpr uint32_t kXBox = kTiles * 8 * 128;      // 64 values of each row
  static constexpr uint32_t kStage = kCodeBoxes * kCodeBox + kXBoxes * kXBox;
  static constexpr uint32_t kSums = kWarpsK * kQ4TileN * kTiles * 8 * 4;
  static constexpr uint32_t kTable = (sizeof(Q4Tables) + 15) / 16 * 16 + kWarps * 2 * 16;
  // Two CTAs per SM, with as many stages as there is room for.  (A single unit's sums take
  // the ring's place.)
  static constexpr int kCtas = 2;
  static constexpr uint32_t kRest = (kExperts ? kSums + kTable : 0) + 256 + 1024;
  static constexpr int S = (233472 / kCtas - 1024 - kRest) / kStage;
  static constexpr uint32_t kSmem = S * kStage + kRest;
  static_assert(kSums <= S * kStage && S >= 2 && kSmem <= 232448, "shared memory");
};

template <int S>
struct alignas(8) Barriers {
  uint64_t full[S];
  uint64_t empty[S];
  int abort;
};

template <typename T>
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  if constexpr (__is_same(T, __half))
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A zero as what is added to codes: in FP16 -(1024 + z) and -(64 + z), in BF16 -z / 64.
template <typename T>
struct Zero {
  uint32_t a, b;
  __device__ __forceinline__ explicit Zero(uint32_t z) {
    if constexpr (__is_same(T, __half)) {
      a = 0xE400E400u + z * 0x00010001u;
      b = 0xD400D400u + z * 0x00100010u;
    } else {
      const float v = (float)z * -0x1p-6f;
      a = pack2<T>(v, v);
      b = 0;
    }
  }
};

// The pairs (0, 4), (1, 5), (2, 6), (3, 7) of a word's codes, less their zero, over
// kQ4Value.  FP16: a code in the low mantissa bits of 1024 is that plus the code, and four
// bits further up 1024 + 16 q (the known conversion of small integers by a magic number, for
// 4-bit weights in Kim, Henry, Fahim and Hassan Awadalla, "Who Says Elephants Can't Run",
// 2022).  BF16 has no room for the latter; but the integer n in the
// low eight bits of a BF16 number is n 2^-133, whether it is subnormal (n < 128) or not, and
// the multiplication with 2^127, or 2^123 for a code four bits further up, is exact.
template <typename T>
__device__ __forceinline__ void codes_less_zero(uint32_t w, const Zero<T>& z, uint32_t (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = w >> (8 * i);
    if constexpr (__is_same(T, __half)) {
      v[2 * i] = fma_x2<T>(and_or(x, 0x000F000Fu, 0x64006400u), 0x3C003C00u, z.a);
      v[2 * i + 1] = fma_x2<T>(and_or(x, 0x00F000F0u, 0x64006400u), 0x2C002C00u, z.b);   // 1/16
    } else {
      v[2 * i] = fma_x2<T>(x & 0x000F000Fu, 0x7F007F00u, z.a);          // 2^127
      v[2 * i + 1] = fma_x2<T>(x & 0x00F000F0u, 0x7D007D00u, z.a);      // 2^123
    }
  }
}

// A barrier of the warps that multiply: whether `b` holds in any thread.
__device__ __forceinline__ bool products_any(bool b) {
  int any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "bar.red.or.pred p, 1, %2, q;\n\tselp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(any)
      : "r"((int)b), "n"(32 * kWarps)
      : "memory");
  return any != 0;
}

// kRun: steps of 32 terms that have one scale (1, 2, or 4: a warp's slice of a stage, where
// groups are a multiple of 128).
template <typename T, int kTiles, int kRun, bool kExperts>
__global__ void __launch_bounds__(kThreads, Layout<kTiles, kExperts>::kCtas)
    q4_few_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmX,
                  const Q4FewParams p) {
  using L = Layout<kTiles, kExperts>;
  constexpr int S = L::S;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* const base = align_smem_1024(smem_raw);
  float* const sums = reinterpret_cast<float*>(base + (kExperts ? S * L::kStage : 0));
  // (kExperts:) each warp's unit and the next, the tables.
  int4* const entered = reinterpret_cast<int4*>(base + S * L::kStage + L::kSums);
  Q4Tables& tables = *reinterpret_cast<Q4Tables*>(entered + 2 * kWarps);
  __shared__ Q4Unit s_unit;
  auto* bars = reinterpret_cast<Barriers<S>*>(base + L::kSmem - 256 - 1024);
  static_assert(sizeof(Barriers<S>) <= 256, "barrier block must fit its reserved space");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;
  const unsigned first = blockIdx.x / (unsigned)p.split, step = gridDim.x / (unsigned)p.split;
  const Q4Walk walk0(kExperts ? p.N : 1, kQ4TileN, first, step);     // (kExperts)
  const int nk = (p.K + kQ4BK - 1) / kQ4BK;
  const int kb = (int)((long long)rank * nk / p.split);
  const int ke = (int)((long long)(rank + 1) * nk / p.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&bars->full[s]), 1);
      mbar_init(smem_u32(&bars->empty[s]), kWarps);
    }
    bars->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmX);
  }
  wait_prior_grids();
  allow_dependent_grids();
  Q4Unit unit0{0, 0, p.rows, (int)first * kQ4TileN, true};
  if constexpr (kExperts) {
    if (warp == 0) {
      Q4Unit w = q4_tables(p, tables, walk0.slot);
      w.n0 = walk0.n * kQ4TileN;
      if (lane == 0) s_unit = w;
    }
  }
  __syncthreads();
  if constexpr (kExperts) unit0 = s_unit;
  if (!unit0.real) return;   // (the same in all of a cluster)
  const bool loop = kExperts && p.split == 1;

  constexpr int kPlane = kQ4TileN * kTiles * 8;
  T* const Y = static_cast<T*>(p.Y);
  // The ranges of K in order: to Y, or into the first where a cluster adds on.  (Experts: by
  // the warps that multiply.)
  auto add_ranges = [&](int lo, int hi, int n0) {
    const int values = (hi - lo) * kQ4TileN;
    for (int i = threadIdx.x; i < values; i += kExperts ? 32 * kWarps : kThreads) {
      float v = sums[i];
#pragma unroll
      for (int j = 1; j < kWarpsK; ++j) v += sums[j * kPlane + i];
      const int n = n0 + i % kQ4TileN;
      if (p.split > 1)
        sums[i] = v;
      else if (n < p.N)
        Y[(long long)(lo + i / kQ4TileN) * p.ldy + n] = from_f32_any<T>(v * kQ4Value<T>);
    }
  };
  uint32_t issued = 0;
  if (warp == kWarps) {
    if (elect_one()) {
      // ---------------------------------------------- loads
      RingPos<S> pos;
      bool ok = true;
      Q4Unit unit = unit0;
      for (Q4Walk walk = walk0; ok && unit.real;) {
        for (int kt = kb; kt < ke; ++kt, pos.next()) {
          ok = role_wait(smem_u32(&bars->empty[pos.slot]), pos.parity ^ 1u, p.fault, p.timeout_ns,
                         &bars->abort, kFaultTcProducerWait, true);
          if (!ok) break;
          const uint32_t st = smem_u32(base + pos.slot * L::kStage);
          const uint32_t full = smem_u32(&bars->full[pos.slot]);
          mbar_arrive_expect_tx(full, L::kStage);
#pragma unroll
          for (int j = 0; j < kCodeBoxes; ++j)
            tma_load_3d(st + j * kCodeBox, &tmQ, full, (kt * kQ4BK + j * 256) / 2, unit.n0,
                        unit.expert);
#pragma unroll
          for (int j = 0; j < kXBoxes; ++j)
            tma_load_2d(st + kCodeBoxes * kCodeBox + j * L::kXBox, &tmX, full, kt * kQ4BK + j * 64,
                        unit.lo);
          ++issued;
        }
        if (!loop) break;
        walk.next();
        unit = q4_unit(p, tables, walk, kQ4TileN);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ products
    const int wn = warp / kWarpsK, wk = warp % kWarpsK;
    const int g = lane >> 2, t = lane & 3;
    const int groups = q4_groups(p.K, p.group);
    constexpr int kSteps = kSliceK / 32, kRuns = kSteps / kRun;
    // This lane's row of W, whose scales and zeros it reads for the warp: a group's
    // are stored together (with a row's stored together each lane read a line of its
    // own: 13.3 us at 8192 x 8192 with groups of 128, 28.8 with 32).
    const uint16_t* scales;
    const unsigned char* zeros;
    bool real;
    auto row_of = [&](const Q4Unit& w) {
      const int row = w.n0 + wn * 32 + lane;
      const long long at = (long long)w.expert * groups * p.N + row;
      scales = static_cast<const uint16_t*>(p.scales) + at;
      zeros = p.zeros != nullptr ? p.zeros + at : nullptr;
      real = row < p.N;
    };
    // The scales and zeros of a stage's slice, read a stage ahead and left as they
    // come: a conversion would wait for them at once.  `at`, `pos`: group of a
    // slice's first step, and its place in it.
    uint16_t sc[kRuns];
    unsigned char zr[kRuns];
    const int far_at = kQ4BK / p.group, far_pos = kQ4BK % p.group;
    const int first_at = (kb * kQ4BK + wk * kSliceK) / p.group;
    const int first_pos = (kb * kQ4BK + wk * kSliceK) % p.group;
    int at = first_at, pos = first_pos;
    auto read_scales = [&](int kt, int at, int pos) {
#pragma unroll
      for (int i = 0; i < kRuns; ++i) {
        const bool ok =
            real && kt < ke && kt * kQ4BK + wk * kSliceK + i * kRun * 32 < p.K;
        const long long to = (long long)at * p.N;
        sc[i] = ok ? scales[to] : (uint16_t)0;
        zr[i] = ok && zeros != nullptr ? zeros[to] : (unsigned char)8;
        if ((pos += kRun * 32) == p.group) pos = 0, ++at;
      }
    };
    row_of(unit0);
    read_scales(kb, at, pos);
    Q4Walk walk = walk0;
    int expert = unit0.expert;
    uint32_t turn = 0;        // (of a unit)
    auto enter = [&](const Q4Unit& w, uint32_t turn) {
      if (kExperts && lane == 0)
        entered[warp * 2 + (turn & 1)] = make_int4(w.lo, w.hi, w.n0, 0);
    };
    enter(unit0, 0);
    // Chunks of 16 bytes in 128-byte rows are swizzled by the row.  (An 8-row tile of
    // X has its rows in the order 0, 4, 1, 5, 2, 6, 3, 7: eight lanes with two rows'
    // four chunks then read 128 different bytes.)
    const int xr = (g >> 1) | ((g & 1) << 2);
    uint32_t q_at[kSteps], x_at[2];
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
      q_at[i] = (wk >> 1) * kCodeBox + (wn * 32 + g) * 128 + t * 4 +
                ((((wk & 1) * 4 + i) ^ g) << 4);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      x_at[i] = kCodeBoxes * kCodeBox + wk * 2 * L::kXBox + xr * 128 + (((i * 4 + t) ^ xr) << 4);
    RingPos<S> ring;
    bool ok = true;
    bool more = true;
    for (; more; ++turn) {
      float acc[2][kTiles][4];
#pragma unroll
      for (int i = 0; i < 2 * kTiles * 4; ++i) (&acc[0][0][0])[i] = 0.f;
      more = false;
      for (int kt = kb; kt < ke; ++kt, ring.next()) {
        float s[kRuns];
        uint32_t z[kRuns];
#pragma unroll
        for (int i = 0; i < kRuns; ++i) {
          s[i] = elem_to_f32<T>(__builtin_bit_cast(T, sc[i]));
          z[i] = zr[i] & 15u;
        }
        at += far_at;
        if ((pos += far_pos) >= p.group) pos -= p.group, ++at;
        int k_far = kt + 1;
        if (loop && k_far == ke) {
          walk.next();
          const Q4Unit next = q4_unit_by_warp(p, tables, walk, kQ4TileN, expert);
          if (next.real) {
            row_of(next);
            enter(next, turn + 1);
            expert = next.expert;
            more = true, k_far = kb, at = first_at, pos = first_pos;
          }
        }
        read_scales(k_far, at, pos);
        ok = role_wait_lanes(smem_u32(&bars->full[ring.slot]), ring.parity, p.fault, p.timeout_ns,
                             &bars->abort, kFaultTcMmaWait);
        if (!ok) break;
        const uint32_t st = smem_u32(base) + ring.slot * L::kStage;
        // (Past K, X is zeros and the codes stand for finite values.)
        uint32_t w[kSteps][4];
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            w[i][r] = ld_shared_u32(st + q_at[i] + r * 8 * 128);
        float part[2][kTiles][4];
        Zero<T> zero[4] = {Zero<T>(0), Zero<T>(0), Zero<T>(0), Zero<T>(0)};
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          if (i % kRun == 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              zero[r] = Zero<T>(__shfl_sync(0xffffffffu, z[i / kRun], r * 8 + g));
#pragma unroll
            for (int e = 0; e < 2 * kTiles * 4; ++e) (&part[0][0][0])[e] = 0.f;
          }
          uint32_t v[4][4];
#pragma unroll
          for (int r = 0; r < 4; ++r) codes_less_zero<T>(w[i][r], zero[r], v[r]);
#pragma unroll
          for (int m = 0; m < kTiles; ++m) {
            const uint4 x = ld_shared_v4(st + x_at[i & 1] + (i >> 1) * L::kXBox + m * 1024);
            const uint32_t b0 = __byte_perm(x.x, x.z, 0x5410), b1 = __byte_perm(x.x, x.z, 0x7632);
            const uint32_t b2 = __byte_perm(x.y, x.w, 0x5410), b3 = __byte_perm(x.y, x.w, 0x7632);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a0[4] = {v[2 * h][0], v[2 * h + 1][0], v[2 * h][1], v[2 * h + 1][1]};
              const uint32_t a1[4] = {v[2 * h][2], v[2 * h + 1][2], v[2 * h][3], v[2 * h + 1][3]};
              mma_16816<T>(part[h][m], a0, b0, b1);
              mma_16816<T>(part[h][m], a1, b2, b3);
            }
          }
          if (i % kRun == kRun - 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float lo = __shfl_sync(0xffffffffu, s[i / kRun], h * 16 + g);
              const float hi = __shfl_sync(0xffffffffu, s[i / kRun], h * 16 + 8 + g);
#pragma unroll
              for (int m = 0; m < kTiles; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  acc[h][m][e] = fmaf(e < 2 ? lo : hi, part[h][m][e], acc[h][m][e]);
            }
          }
        }
        // The proxy fence waits for the loads above: without it TMA has been seen to
        // refill the stage before the last of them had read it.
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->empty[ring.slot]));
      }
      // sums[wk][row of X][row of W]: where the stages were, or once the last unit's have
      // been read.
      if (!kExperts || turn != 0) asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory");
      float* const to = sums + wk * kPlane + wn * 32;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < kTiles; ++m)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            to[(m * 8 + t + 4 * (e & 1)) * kQ4TileN + h * 16 + (e >> 1) * 8 + g] = acc[h][m][e];
      if constexpr (!kExperts) break;
      // (All of them go on or none.)
      if (products_any(!ok)) break;
      const int4 unit = entered[warp * 2 + (turn & 1)];
      add_ranges(unit.x, unit.y, unit.z);
    }
  }
  __syncthreads();
  if (warp == kWarps && elect_one() && bars->abort) {
    // Let the copies in flight land.
    for (uint32_t it = issued > (uint32_t)S ? issued - S : 0; it < issued; ++it)
      if (!mbar_wait_bounded(smem_u32(&bars->full[it % S]), (it / S) & 1u, p.timeout_ns,
                             nullptr)) {
        raise_fault(p.fault, kFaultDrainWait);
        break;
      }
  }
  if constexpr (!kExperts) add_ranges(unit0.lo, unit0.hi, unit0.n0);
  if (p.split > 1) {
    // This CTA's part of the tile over the cluster.  (Only what is stored is read: see
    // cluster_arrive_relaxed().)
    cluster_sync_all();
    const Q4Unit unit = unit0;
    const int values = (unit.hi - unit.lo) * kQ4TileN;
    for (int i = rank * kThreads + threadIdx.x; i < values; i += p.split * kThreads) {
      const int n = unit.n0 + i % kQ4TileN;
      if (n >= p.N) continue;
      const uint32_t at = smem_u32(sums + i);
      float v = 0.f;
      for (int r = 0; r < p.split; ++r) v += ld_cluster_f32(mapa_shared(at, (uint32_t)r));
      Y[(long long)(unit.lo + i / kQ4TileN) * p.ldy + n] = from_f32_any<T>(v * kQ4Value<T>);
    }
    // Nobody leaves while its sums may still be read.
    cluster_arrive_relaxed();
    cluster_wait();
  }
}

template <typename T, int kTiles, int kRun, bool kExperts>
cudaError_t launch_tiles(const Q4FewParams& p, const CUtensorMap* tmQ, const CUtensorMap* tmX,
                         cudaStream_t stream) {
  using L = Layout<kTiles, kExperts>;
  auto kernel = q4_few_kernel<T, kTiles, kRun, kExperts>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = mx_allow_smem(kernel, L::kSmem, &done);
  if (e != cudaSuccess) return e;
  const long long units = ((long long)p.N + kQ4TileN - 1) / kQ4TileN * p.slots;
  const long long ctas = kExperts && units > p.max_ctas ? p.max_ctas : units;
  return launch_gemm_kernel_clusters((unsigned)p.split, kernel, dim3((unsigned)(ctas * p.split)),
                                     dim3(kThreads), L::kSmem, stream, *tmQ, *tmX, p);
}

template <typename T, int kTiles, bool kExperts>
cudaError_t launch_run(const Q4FewParams& p, const CUtensorMap* q, const CUtensorMap* x,
                       cudaStream_t stream) {
  if (p.group % 128 == 0) return launch_tiles<T, kTiles, 4, kExperts>(p, q, x, stream);
  return p.group % 64 == 0 ? launch_tiles<T, kTiles, 2, kExperts>(p, q, x, stream)
                           : launch_tiles<T, kTiles, 1, kExperts>(p, q, x, stream);
}

template <typename T>
cudaError_t launch_typed(const Q4FewParams& p, const CUtensorMap* q, const CUtensorMap* x,
                         cudaStream_t stream) {
  if (p.experts != 0) return launch_run<T, 1, true>(p, q, x, stream);
  return p.tile_rows == 8 ? launch_run<T, 1, false>(p, q, x, stream)
                          : launch_run<T, 2, false>(p, q, x, stream);
}

}  // namespace

int q4_few_clusters(int split) {
  static std::atomic<int> known[9][64];
  return clusters_at_once(q4_few_kernel<__half, 1, 4, false>, (unsigned)split, kThreads,
                          Layout<1, false>::kSmem, known[split]);
}

cudaError_t launch_q4_few(int dtype, const Q4FewParams& p, const CUtensorMap* tmQ,
                          const CUtensorMap* tmX, cudaStream_t stream) {
  return dtype == 1 ? launch_typed<__half>(p, tmQ, tmX, stream)
                    : launch_typed<__nv_bfloat16>(p, tmQ, tmX, stream);
}

}  // namespace dgemm
