// The work of the grouped kernels' CTA pairs, from offsets that only the device
// knows: units of C, which the pairs take in rounds, and their draining.
//
// A group's rows are cut into equal tiles of at most 256 (few rows: 64), a multiple of 32
// (1342 rows: six of 224 rather than five of 256 and one of 62), so that the units of a
// round end together: 8192 rows of 8 experts, 4096 x 4096, 167 -> 161 us.  (Groups taken in
// the order of their units' cost changed nothing.  Where there are more units than pairs,
// ranges of units cut along K, one for each pair, whose pieces meet through a workspace, were
// slower in every case: storing and adding the pieces took 8 to 10 us at the end, the last
// round that is not full 4 to 8.)
#pragma once

#include "group.h"
#include "mx.cuh"

namespace dgemm {

constexpr int kGroupEpiWarps = 8;

// A unit: rows [row, row_end) of C (at most a tile; weights: of C[g]) by the 256
// columns from col; the sum's k-tiles are nk, from row k0 of the operands and up
// to k_end (weights; products: from column 0 up to K).
struct GroupUnit {
  int g, row, row_end, col;
  int nk, k0, k_end;
  int mma_rows;             // rows rounded up to the MMA's steps of 32
};

// The groups' ends in order, 32 at a time, by a warp: offsets that decrease or leave 0 ..
// rows are moved to the nearest that do not.  (No offsets: one group has all rows.)
struct GroupEnds {
  const int* offsets;
  int rows;
  __device__ __forceinline__ int clamp(int v) const { return min(max(v, 0), rows); }
  __device__ __forceinline__ int first() const {
    return offsets == nullptr ? 0 : clamp(offsets[0]);
  }
  __device__ __forceinline__ bool first_is_bad() const {
    return offsets != nullptr && offsets[0] != clamp(offsets[0]);
  }
  // End of group i (of `groups`; lanes past them: the last one's), and where it begins;
  // *last: where the lanes' first group begins, then where their last ends.
  __device__ __forceinline__ int next(int i, int groups, int* last, int* before,
                                      bool* bad) const {
    const int lane = threadIdx.x & 31;
    const int raw = i >= groups ? 0 : (offsets == nullptr ? rows : offsets[i + 1]);
    int v = i >= groups ? *last : clamp(raw);
    const int own = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, v, d);
      if (lane >= d) v = max(v, o);
    }
    v = max(v, *last);
    *bad |= i < groups && (own != raw || v != own);
    const int o = __shfl_up_sync(0xffffffffu, v, 1);
    *before = lane == 0 ? *last : o;
    *last = __shfl_sync(0xffffffffu, v, 31);
    return v;
  }
};

struct GroupTables {
  int start[kGroupMaxGroups + 1];        // first rows of the groups, in order
  int unit0[kGroupMaxGroups + 1];        // their first units
  short tile[kGroupMaxGroups];           // rows of their tiles
  int units;
};

// Rows of a group's tiles of at most kRows (m > 0).
template <int kRows>
__device__ __forceinline__ int group_tile_rows(int m) {
  const int tiles = (m + kRows - 1) / kRows;
  return ((int)((unsigned)(m + tiles - 1) / (unsigned)tiles) + 31) & ~31;
}
__device__ __forceinline__ int group_k_tiles(int terms) { return (terms + kGroupBK - 1) / kGroupBK; }

// The last group g in [0, groups) with first[g] <= x.
template <typename V>
__device__ __forceinline__ int group_find(const V* first, int groups, V x) {
  int lo = 0, hi = groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// The tables, by one warp.  kRows: most rows of a tile.
template <int kKind, int kRows>
__device__ __forceinline__ void group_tables(const GroupParams& p, GroupTables& t) {
  const int lane = threadIdx.x & 31;
  const int tiles_n = (p.N + kGroupTile - 1) / kGroupTile;
  const GroupEnds ends{p.offsets, p.rows};
  int units = 0;
  int last = ends.first();
  bool bad = ends.first_is_bad();
  for (int base = 0; base < p.first_group + p.groups; base += 32) {
    const int i = base + lane, g = i - p.first_group;
    int before;
    const int end = ends.next(i, p.first_group + p.groups, &last, &before, &bad);
    const bool is = g >= 0 && g < p.groups;
    if (is) t.start[g] = before;
    if (kKind != kGroupWeights) {
      const int m = end - before, mine = is ? (m + kRows - 1) / kRows * tiles_n : 0;
      int n = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, n, d);
        if (lane >= d) n += o;
      }
      if (is) t.unit0[g] = units + n - mine;
      if (is && m > 0) t.tile[g] = (short)group_tile_rows<kRows>(m);
      units += __shfl_sync(0xffffffffu, n, 31);
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0 && blockIdx.x == 0)
    raise_fault(p.fault, kFaultGroupOffsets);
  if (lane == 0) {
    t.start[p.groups] = last;
    t.unit0[p.groups] = units;
    t.units = kKind == kGroupWeights ? p.groups * p.per_group : units;
  }
}

template <int kKind, int kRows>
__device__ __forceinline__ GroupUnit group_unit(int u, const GroupParams& p,
                                                const GroupTables& t) {
  GroupUnit w;
  int tm, tn;
  if constexpr (kKind == kGroupWeights) {
    w.g = u / p.per_group;
    // (Groups of 16 tiles along C's columns share the operands in L2.)
    grouped_tile(u - w.g * p.per_group, (p.N + kGroupTile - 1) / kGroupTile,
                 (p.M + kRows - 1) / kRows, 16, tn, tm);
    w.row = tm * kRows;
    w.row_end = min(w.row + kRows, p.M);
    w.k0 = t.start[w.g];
    w.k_end = t.start[w.g + 1];
    w.nk = p.K == 0 ? 0 : group_k_tiles(w.k_end - w.k0);
  } else {
    w.g = group_find(t.unit0, p.groups, u);
    const int first = t.start[w.g], rows = t.start[w.g + 1] - first, tile = t.tile[w.g];
    grouped_tile(u - t.unit0[w.g], (rows + kRows - 1) / kRows,
                 (p.N + kGroupTile - 1) / kGroupTile, 16, tm, tn);
    w.row = first + tm * tile;
    w.row_end = min(w.row + tile, first + rows);
    w.k0 = 0;
    w.k_end = p.K;
    w.nk = group_k_tiles(p.K);
  }
  w.col = tn * kGroupTile;
  w.mma_rows = (w.row_end - w.row + 31) & ~31;
  return w;
}

// First k-tile of a part of a unit's nk (at most 2^24).
__device__ __forceinline__ int group_part_first(int nk, int part, const GroupParams& p) {
  return nk * part >> p.log_parts;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// ------------------------------------------------------------ draining

// Drains a cluster's units (each CTA, kGroupEpiWarps warps): warp `ew` takes TMEM lanes
// 32 (ew % 4) .. + 31 (columns of C) and every other 32 rows.  Where pairs share a unit
// (p.log_parts > 0: no more than one for the cluster), their sums go to shared memory, `sums`,
// row by row of the CTA's 128 columns.
template <typename TC, int kKind, int kRows, typename Bars>
__device__ __forceinline__ void group_epilogue(const GroupParams& p, const GroupTables& t,
                                               Bars* bars, uint32_t tmem_base, uint32_t crank,
                                               int ew, int cluster, int clusters, float* sums) {
  const int lane = threadIdx.x & 31;
  const int q = ew & 3, half = ew >> 2;
  constexpr bool kWeights = kKind == kGroupWeights;
  const uint32_t rank = crank & 1u, leader = crank & ~1u;
  const int part = (int)(crank >> 1);
  const bool pairs = (reinterpret_cast<uintptr_t>(p.C) & 3u) == 0 && ((p.ldc | p.N) & 1) == 0 &&
                     (p.stride_c & 1) == 0;
  uint32_t seg = 0;
  bool ok = true;
  for (int u = cluster; u < t.units; u += clusters) {
    const GroupUnit w = group_unit<kKind, kRows>(u, p, t);
    const int chunks = w.mma_rows / 32;
    constexpr int kChunks = kRows / 64;                    // of 32 rows, this warp's
    float acc[32 * kChunks];
#pragma unroll
    for (int j = 0; j < 32 * kChunks; ++j) acc[j] = 0.f;
    const int k_first = group_part_first(w.nk, part, p);
    const int k_last = group_part_first(w.nk, part + 1, p);
    for (int k0 = k_first; k0 < k_last; k0 += p.seg, ++seg) {
      const uint32_t b = seg & 1;
      ok = role_wait_lanes(smem_u32(&bars->acc_full[b]), (seg >> 1) & 1u, p.fault, p.timeout_ns,
                           &bars->abort, kFaultTcEpilogueWait, false, false);
      if (!ok) break;
      tc_fence_after();
      const uint32_t ta = tmem_base + ((uint32_t)(q * 32) << 16) + b * 256;
#pragma unroll
      for (int c = 0; c < 2 * kChunks; ++c) {
        const int chunk = 2 * (c >> 1) + half;
        if (chunk < chunks) {
          uint32_t r[16];
          tmem_ld16(ta + chunk * 32 + (c & 1) * 16, r);
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[c * 16 + j] += __uint_as_float(r[j]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_any_cta(mapa_shared(smem_u32(&bars->acc_empty[b]), leader));
    }
    if (!ok) break;
    if (p.log_parts > 0) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const int chunk = 2 * c + half;
        if (chunk < chunks) {
          float* const to = sums + chunk * 32 * 128 + q * 32 + lane;
#pragma unroll
          for (int j = 0; j < 32; ++j) to[j * 128] = acc[c * 32 + j];
        }
      }
      break;
    }
    const int col = w.col + (int)rank * 128 + q * 32 + lane;
    TC* c_out = static_cast<TC*>(p.C) + (kWeights ? w.g * p.stride_c : 0);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const int chunk = 2 * c + half;
      if (chunk < chunks)
        store_piece<TC>(acc + c * 32, c_out, p.ldc, w.row_end, p.N, w.row + chunk * 32, col, pairs,
                        p.alpha, p.beta);
    }
  }
}

}  // namespace dgemm
