// Device helpers of the microscaled (MX) kernels: element conversions, block
// scales, tcgen05 block-scaled MMA and scale copies, bounded role waits.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "mx.h"
#include "ptx.cuh"
#include "tcgen05.cuh"

namespace dgemm {

// Byte offset of the scale of (row, block) in an array whose rows have
// `tiles` tiles of scales.
__host__ __device__ __forceinline__ long long mx_scale_offset(int row, int block, int tiles) {
  return ((long long)(row >> 7) * tiles + (block >> 2)) * kMxTileBytes + (row & 31) * 16 +
         ((row >> 5) & 3) * 4 + (block & 3);
}

// Scale byte of a block whose largest |x| has the FP32 bits `amax`:
// floor(log2) - emax + 127, clamped to [0, 254]; 255 for an infinity or NaN.
// (The exponent field of a subnormal is 0, which clamps to 0 as well.)
template <int kFmt>
__device__ __forceinline__ unsigned mx_scale_byte(unsigned amax) {
  const int e = (int)(amax >> 23);
  if (e == 255) return 255u;
  constexpr int emax = kFmt == GEMM_MXFP4 ? 2 : 0;
  return (unsigned)(e > emax ? e - emax : 0);
}

// 2^(127 - s), the exact reciprocal of the scale s (0 .. 254; for 255, whose
// codes are zeros, 0).
__device__ __forceinline__ float mx_inverse_scale(unsigned s) {
  const unsigned bits = s < 254u ? (254u - s) << 23 : (s == 254u ? 0x00400000u : 0u);
  return __uint_as_float(bits);
}

// 2^(s - 127); NaN for 255.
__device__ __forceinline__ float mx_scale_value(unsigned s) {
  const unsigned bits = s == 0u ? 0x00400000u : (s == 255u ? 0x7FC00000u : s << 23);
  return __uint_as_float(bits);
}

// Eight values, already divided by their scale, as E2M1 codes (value j in
// bits 4j .. 4j + 3), rounded to nearest even and saturated to +-6.
__device__ __forceinline__ unsigned e2m1x8(const float (&v)[8]) {
  unsigned r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Eight values, already divided by their scale, as MXINT8 codes: v * 64
// rounded to nearest even (adding 1.5 * 2^23 leaves the integer in the low
// mantissa bits).  Only values of 127.5 / 64 or more would round past +-127;
// `clamp` says whether the block has any (its largest shows that).
__device__ __forceinline__ uint2 int8x8(float (&v)[8], bool clamp) {
  if (clamp) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fminf(fmaxf(v[i], -1.984375f), 1.984375f);
  }
  unsigned b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(fmaf(v[i], 64.f, 12582912.f));
  uint2 r;
  r.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
  r.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
  return r;
}
__device__ __forceinline__ bool int8_clamps(unsigned amax, float inv) {
  return __uint_as_float(amax) * inv >= 1.9921875f;
}

// Eight E2M1 codes as FP32 values (without their scale).
__device__ __forceinline__ void e2m1x8_to_f32(unsigned codes, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    unsigned h;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}"
        : "=r"(h)
        : "r"(codes >> (8 * j)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * j] = f.x;
    v[2 * j + 1] = f.y;
  }
}
// Four MXINT8 codes (one word) as FP32 values (without their scale):
// 0x4B000000 + u is 2^23 + u; u = c + 128.
__device__ __forceinline__ void int8x4_to_f32(unsigned w, float* v) {
  const unsigned u = w ^ 0x80808080u;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + j)) - 8388736.f) * 0.015625f;
}

template <typename T>
__device__ __forceinline__ float to_f32_any(T v) {
  if constexpr (sizeof(T) == 4)
    return v;
  else
    return elem_to_f32<T>(v);
}
template <typename T>
__device__ __forceinline__ T from_f32_any(float v) {
  if constexpr (sizeof(T) == 4)
    return v;
  else if constexpr (__is_same(T, __half))
    return __float2half_rn(v);
  else
    return __float2bfloat16_rn(v);
}

// Eight consecutive elements of type T, 16-byte aligned.
template <typename T>
__device__ __forceinline__ void load8(const T* src, float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = *reinterpret_cast<const float4*>(src);
    const float4 b = *reinterpret_cast<const float4*>(src + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(src);
    const unsigned w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = pair_to_f32<T>(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}
__device__ __forceinline__ unsigned abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// ------------------------------------------------------------ tcgen05, block scaled

// Shared-memory matrix descriptors in two words.  The high word (stride
// between 8-row groups, version, swizzle) is the same for all of a kernel's
// tiles, and the low one (address, leading offset) of a tile further along
// differs by a plain addition of its distance in 16-byte units: one
// instruction per operand of an MMA, which the issuing thread, alone in its
// warp, can afford.
constexpr uint32_t kDescHi128B = (1024u >> 4) | (1u << 14) | (2u << 29);   // 128-byte swizzle
constexpr uint32_t kDescHiPlain = (128u >> 4) | (1u << 14);                // 8 rows of 16 bytes
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16);
}

// Instruction descriptor of kind::mxf4: E2M1 operands (K-major), E8M0
// scales; M = m, N = n, and the byte (0 or 2) of the scale words at which
// the step's two scales start.
__host__ __device__ constexpr uint32_t instr_desc_mx4(uint32_t m, uint32_t n, uint32_t sf) {
  return (sf << 4)                 // B scale byte
         | (1u << 7)               // A format: E2M1
         | (1u << 10)              // B format: E2M1
         | ((n >> 3) << 17)
         | (1u << 23)              // scale format: E8M0
         | ((m >> 4) << 24)
         | (sf << 29);             // A scale byte
}

// 16-deep kind::f16 MMA step of a CTA pair (see mma_f16_pair), 128-byte
// swizzled operands.
__device__ __forceinline__ void mma_f16_pair_lo(uint32_t d_tmem, uint32_t alo, uint32_t blo,
                                                uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(alo), "r"(blo), "r"(kDescHi128B), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 64-deep block-scaled MMA step of a CTA pair; each CTA's tensor memory holds
// the scales of its own rows of A and of all of B.
__device__ __forceinline__ void mma_mx4_pair(uint32_t d_tmem, uint32_t alo, uint32_t blo,
                                             uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %7, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %4, [%5], "
      "[%6], p;\n\t}" ::"r"(d_tmem),
      "r"(alo), "r"(blo), "r"(kDescHi128B), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Registers to 16 or 32 consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Untiled bulk copy global -> shared; addresses and size multiples of 16.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// True in one lane of a converged warp, always the same one (so that a later
// tcgen05.commit covers what the role issued).  Roles of a single thread branch on
// this rather than on the lane's number: the compiler then knows that one
// thread runs them and keeps addresses and descriptors in uniform registers,
// where TMA and tcgen05 instructions want them (dX 4096^3 86.6 -> 80.5 us, the
// 4-bit product 28.4 -> 27.0).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// ------------------------------------------------------------ role waits

// A role's bounded wait by one thread; on giving up records the fault (once
// per CTA) and raises the CTA's abort flag.  `spin`: no suspend hint.  The
// clock is first read after a number of tries, because reading %globaltimer
// takes longer than most of these waits last.
__device__ __forceinline__ bool role_wait(uint32_t bar, uint32_t parity, unsigned* fault,
                                          unsigned long long timeout_ns, int* abort,
                                          unsigned code, bool spin) {
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (spin ? mbar_try_wait(bar, parity) : mbar_try_wait_suspend(bar, parity, 10000u)) return true;
    if ((it & 255u) == 0) {
      const uint64_t now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (*(volatile int*)abort || now - t0 > timeout_ns) {
        if (!*(volatile int*)abort) raise_fault(fault, code);
        *(volatile int*)abort = 1;
        return false;
      }
    }
  }
}
// The same by a warp, each lane polling (`ready`: what an earlier try of the
// lane gave).  One lane polling while the others wait for its answer is much
// slower where a warp waits for every stage (dX 4096^3 152 against 89 us) and
// still shows where it waits once per tile (89.2 against 86.5 us).
__device__ __forceinline__ bool role_wait_lanes(uint32_t bar, uint32_t parity, unsigned* fault,
                                                unsigned long long timeout_ns, int* abort,
                                                unsigned code, bool ready = false,
                                                bool spin = true) {
  return __all_sync(0xffffffffu,
                    ready || role_wait(bar, parity, fault, timeout_ns, abort, code, spin));
}

// Arrives on an mbarrier of any CTA of the cluster (shared::cluster address)
// with the default release at CTA scope.  What the arrivals here hand over
// is read by the asynchronous proxy (after fence.proxy.async by the writer)
// or is tensor memory (after tcgen05 fences); a release at cluster scope
// would wait some 1000 cycles for every earlier access of the thread.
__device__ __forceinline__ void mbar_arrive_any_cta(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Position in a ring of N slots: slot and the parity of its current use.
template <int N>
struct RingPos {
  uint32_t slot = 0, parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

// ------------------------------------------------------------ pair schedule

// Work unit u of a grid of CTA pairs (MxSchedule): tile column tn (256
// columns of C), rows [row0, row0 + rows) of C (rows = 256 or 128), k-tiles
// [kb, ke).
struct MxUnit {
  int tn, row0, rows, kb, ke, slice;
};
__device__ __forceinline__ MxUnit mx_unit(int u, const MxSchedule& sc, int nk) {
  MxUnit w;
  const int v = u / sc.slices;
  w.slice = u - v * sc.slices;
  w.kb = (int)((long long)w.slice * nk / sc.slices);
  w.ke = (int)((long long)(w.slice + 1) * nk / sc.slices);
  int tm;
  if (sc.by_halves) {
    grouped_tile(v, sc.tiles_n, sc.halves_m, sc.group, w.tn, tm);
    w.rows = kMxPairTile / 2;
    w.row0 = tm * w.rows;
    return w;
  }
  int tile = v, off = 0;
  w.rows = kMxPairTile;
  if (v >= sc.full_tiles) {   // (the second half can lie past M: the roles skip it)
    const int j = v - sc.full_tiles;
    tile = sc.full_tiles + (j >> 1);
    off = (j & 1) * (kMxPairTile / 2);
    w.rows = kMxPairTile / 2;
  }
  grouped_tile(tile, sc.tiles_n, sc.tiles_m, sc.group, w.tn, tm);
  w.row0 = tm * kMxPairTile + off;
  return w;
}

// ------------------------------------------------------------ epilogue

// One thread's 32 FP32 sums to 32 rows of one column of C (c: the first
// row's element; rows_left may be below 32 or even negative):
// C := alpha * sum + beta * C.  A warp's lanes hold 32 consecutive columns,
// so that each store writes one contiguous piece of a row, whatever C's
// alignment.
template <typename T>
__device__ __forceinline__ void store_rows32(const float* v, T* c, long long ldc, int rows_left,
                                             float alpha, float beta) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    if (beta == 0.f) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (8 * g + j < rows_left) c[j * ldc] = from_f32_any<T>(alpha * v[8 * g + j]);
    } else {
      float old[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        old[j] = 8 * g + j < rows_left ? to_f32_any<T>(c[j * ldc]) : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (8 * g + j < rows_left)
          c[j * ldc] = from_f32_any<T>(fmaf(beta, old[j], alpha * v[8 * g + j]));
    }
    c += 8 * ldc;
  }
}

// The same by a whole warp (lanes with consecutive columns, the first even) for
// a 16-bit C whose rows are 4-byte aligned and of even width, without beta:
// lanes swap with their neighbour, so that each stores two columns of every
// other row, in half as many stores.
template <typename T>
__device__ __forceinline__ void store_rows32_pairs(const float* v, T* c, long long ldc,
                                                   int rows_left, bool inside, float alpha) {
  const bool odd = threadIdx.x & 1;
  T* p = c + (odd ? ldc - 1 : 0);
  const int left = inside ? rows_left - (odd ? 1 : 0) : 0;
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    const float got = __shfl_xor_sync(0xffffffffu, odd ? v[j] : v[j + 1], 1);
    const uint32_t w = odd ? pack2<T>(alpha * got, alpha * v[j + 1]) : pack2<T>(alpha * v[j], alpha * got);
    if (j < left) *reinterpret_cast<uint32_t*>(p) = w;
    p += 2 * ldc;
  }
}

// One warp's 32 x 32 piece of C by whichever of the two fits; `pairs`: C is
// 4-byte aligned, ldc and N even.
template <typename T>
__device__ __forceinline__ void store_piece(const float* v, T* C, long long ldc, int M, int N,
                                            int row, int col, bool pairs, float alpha,
                                            float beta) {
  T* c = C + (long long)row * ldc + col;
  if constexpr (sizeof(T) == 2) {
    if (pairs && beta == 0.f) {
      store_rows32_pairs<T>(v, c, ldc, M - row, col < N, alpha);
      return;
    }
  }
  if (col < N) store_rows32<T>(v, c, ldc, M - row, alpha, beta);
}

// 16 consecutive FP32 columns of this thread's TMEM lane, waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Waits for this thread's tcgen05.ld loads into r (see tmem_ld_wait).
__device__ __forceinline__ void tmem_ld_wait32(uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
        "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
        "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
        "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
        "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
      :
      : "memory");
}

}  // namespace dgemm
