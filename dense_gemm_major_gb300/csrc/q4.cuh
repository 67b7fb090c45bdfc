// Device helpers of the kernels with 4-bit weights: tiles of rows, and codes as 16-bit
// integers.
#pragma once

#include "group_sched.cuh"
#include "q4.h"

namespace dgemm {

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* desc, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(desc)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// (a & b) | c
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
template <typename T>
__device__ __forceinline__ uint32_t fma_x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  if constexpr (__is_same(T, __half))
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  else
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
template <typename T>
__device__ __forceinline__ uint32_t mul_x2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (__is_same(T, __half))
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Codes less their zeros are made as multiples of 1 / kQ4Value; results are multiplied by it.
template <typename T>
constexpr float kQ4Value = __is_same(T, __half) ? 1.f : 64.f;

// Volatile, so that no load moves past the arrival that gives its stage back.
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Tile `slot` of the rows, tile_rows each: its expert (-1: there is no such tile) and
// rows [lo, hi).  By one warp.
struct Q4Rows {
  int expert, lo, hi;
};
__device__ __forceinline__ Q4Rows q4_rows_of_slot(int slot, const Q4FewParams& p) {
  Q4Rows r;
  if (p.experts == 0) {
    r.expert = 0;
    r.lo = slot * p.tile_rows;
    r.hi = min(r.lo + p.tile_rows, p.rows);
    return r;
  }
  r.expert = -1, r.lo = r.hi = 0;
  const int lane = threadIdx.x & 31;
  const GroupEnds ends{p.offsets, p.rows};
  int last = ends.first(), tiles = 0;
  bool bad = ends.first_is_bad();
  for (int base = 0; base < p.experts; base += 32) {
    int before;
    const int end = ends.next(base + lane, p.experts, &last, &before, &bad);
    const int mine = (end - before + p.tile_rows - 1) / p.tile_rows;
    int n = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, n, d);
      if (lane >= d) n += o;
    }
    const unsigned here =
        __ballot_sync(0xffffffffu, slot < tiles + n && slot >= tiles + n - mine);
    if (here != 0) {
      const int src = __ffs(here) - 1;
      r.expert = base + src;
      const int first = __shfl_sync(0xffffffffu, tiles + n - mine, src);
      r.lo = __shfl_sync(0xffffffffu, before, src) + (slot - first) * p.tile_rows;
      r.hi = min(r.lo + p.tile_rows, __shfl_sync(0xffffffffu, end, src));
    }
    tiles += __shfl_sync(0xffffffffu, n, 31);
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0 && slot == 0)
    raise_fault(p.fault, kFaultGroupOffsets);
  return r;
}

// The tiles of the rows, tile_rows each, by expert (without experts: one has all rows).
struct Q4Tables {
  int start[kGroupMaxGroups + 1];    // first rows of the experts, in order
  short slot0[kGroupMaxGroups];      // their first tiles
  int slots;
};

// kTileN columns of Y for a tile of rows.
struct Q4Unit {
  int expert, lo, hi;     // its rows [lo, hi)
  int n0;
  bool real;              // there is such a unit
};

// A CTA's units: every gridDim.x-th, a tile's one behind the other.
struct Q4Walk {
  int slot, n;            // tile of rows, of columns
  int tiles_n, d_slot, d_n;
  __device__ __forceinline__ Q4Walk(int N, int tile_n, unsigned first, unsigned step) {
    tiles_n = (int)(((unsigned)N + (unsigned)tile_n - 1) / (unsigned)tile_n);
    slot = (int)(first / (unsigned)tiles_n);
    n = (int)(first - (unsigned)slot * (unsigned)tiles_n);
    d_slot = (int)(step / (unsigned)tiles_n);
    d_n = (int)(step - (unsigned)d_slot * (unsigned)tiles_n);
  }
  __device__ __forceinline__ void next() {
    slot += d_slot;
    if ((n += d_n) >= tiles_n) n -= tiles_n, ++slot;
  }
};

// The tables, and the unit of `slot` among them (n0 is the caller's).  By one warp.
__device__ __forceinline__ Q4Unit q4_tables(const Q4FewParams& p, Q4Tables& t, int slot) {
  const int lane = threadIdx.x & 31, experts = max(p.experts, 1);
  const GroupEnds ends{p.offsets, p.rows};
  Q4Unit w{0, 0, 0, 0, false};
  int last = ends.first(), slots = 0;
  bool bad = ends.first_is_bad();
  for (int base = 0; base < experts; base += 32) {
    const int e = base + lane;
    int before;
    const int end = ends.next(e, experts, &last, &before, &bad);
    const int mine = (end - before + p.tile_rows - 1) / p.tile_rows;
    int n = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, n, d);
      if (lane >= d) n += o;
    }
    const int first = slots + n - mine;
    if (e < experts) {
      t.start[e] = before;
      t.slot0[e] = (short)first;
    }
    const unsigned here = __ballot_sync(0xffffffffu, slot >= first && slot < first + mine);
    if (here != 0) {
      const int src = __ffs(here) - 1;
      w.real = true;
      w.expert = base + src;
      w.lo = __shfl_sync(0xffffffffu, before, src) +
             (slot - __shfl_sync(0xffffffffu, first, src)) * p.tile_rows;
      w.hi = min(w.lo + p.tile_rows, __shfl_sync(0xffffffffu, end, src));
    }
    slots += __shfl_sync(0xffffffffu, n, 31);
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0)
    raise_fault(p.fault, kFaultGroupOffsets);
  if (lane == 0) {
    t.start[experts] = last;
    t.slots = slots;
  }
  return w;
}

__device__ __forceinline__ Q4Unit q4_unit_of(const Q4FewParams& p, const Q4Tables& t,
                                             const Q4Walk& at, int tile_n, int expert) {
  Q4Unit w;
  w.real = at.slot < t.slots;
  w.expert = expert;
  w.lo = t.start[expert] + (at.slot - t.slot0[expert]) * p.tile_rows;
  w.hi = min(w.lo + p.tile_rows, t.start[expert + 1]);
  w.n0 = at.n * tile_n;
  return w;
}
// By one thread.
__device__ __forceinline__ Q4Unit q4_unit(const Q4FewParams& p, const Q4Tables& t,
                                          const Q4Walk& at, int tile_n) {
  return q4_unit_of(p, t, at, tile_n,
                    group_find(t.slot0, max(p.experts, 1), (short)min(at.slot, t.slots)));
}
// By one warp; expert: of an earlier unit.  (A thread's search takes some 900 cycles, which
// loads issued far ahead can bear, but not the warps that convert.)
__device__ __forceinline__ Q4Unit q4_unit_by_warp(const Q4FewParams& p, const Q4Tables& t,
                                                  const Q4Walk& at, int tile_n, int expert) {
  for (int here = 32; here == 32; expert += here) {
    const int e = expert + 1 + (int)(threadIdx.x & 31);
    here = __popc(__ballot_sync(0xffffffffu, e < p.experts && t.slot0[e] <= at.slot));
  }
  return q4_unit_of(p, t, at, tile_n, expert);
}

}  // namespace dgemm
