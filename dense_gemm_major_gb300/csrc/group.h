// Internal interface of the grouped products: the launch functions, called by
// group_api.cu.  Callers use include/dense_gemm_group.h.
#pragma once

#include <atomic>

#include <cuda.h>
#include <cuda_runtime.h>

#include "dense_gemm_group.h"
#include "launch.h"

namespace dgemm {

// The kernel's three forms, by what its MMAs' M side (256 columns of C) and N
// side (up to 256 rows of C) read:
//   forward  B stored N x K, K-major          X, K-major
//   input    B stored K x N, MN-major         X, K-major
//   weights  X, MN-major                      A, MN-major, both over a group's rows
enum GroupKind { kGroupForward = 0, kGroupInput = 1, kGroupWeights = 2 };

constexpr int kGroupTile = 256;       // columns of C, and rows at most, of a CTA pair's unit
constexpr int kGroupBK = 128;
constexpr int kGroupMaxGroups = GEMM_GROUP_MAX_GROUPS;
// Most rows of a product's units, by the rows of a group to expect.  64 / 256, us: 32
// experts of 2048 x 2048: 32 rows 29.6 / 30.9, 256 49.2 / 53.2, 1024 50.2 / 54.9, 2048 51.9 /
// 56.2; 8 of 4096 x 4096: 8 rows 37.5 / 43.4, 512 51.3 / 52.2.  (Each unit reads its
// weights, so that larger groups want larger ones.)
inline int group_unit_rows(int rows, int groups) {
  return rows <= 64ll * groups ? 64 : kGroupTile;
}
// No more units than whole tiles of rows and a ragged one for each group that can have any.
inline long long group_units(int rows, int groups, int N, int tile_rows) {
  return ((long long)rows / tile_rows + (groups < rows ? groups : rows)) *
         ((N + kGroupTile - 1ll) / kGroupTile);
}
// Pairs that share a unit's K (weights: the rows of a group to expect), where there are few
// units.  One / two / four, us:
//   products   8 rows of 1 group, N x K of 1024 x 8192      21.0 / 13.7 / 9.7
//              60 rows of 1, 1024 x 4096                    12.9 / 10.3 / 8.5
//              2 rows of 2, 1024 x 4096                     13.1 / 9.8 / 8.1
//              8 rows of 1, 2560 x 4096                     two 9.6, four 8.2
//              8 rows of 1, 3840 x 4096                     two 10.6, four 9.9
//              500 rows of 1, 1280 x 4096                   two 18.0, four 14.2
//              1 row of 1, 4096 x 4096                      13.5 / 10.6 / 16.7 (a cluster of
//                                        eight CTAs more than run at once)
//              64 rows of 1, 2048 x 2048                    8.9 / 8.4
//              512 rows of 1, 1024 x 8192                   41.5 / 26.9
//   gradients  8192 rows of 1, 256 x 256                    43.7 / 27.7 / 18.5
//              8192 rows of 1, 1024 x 1024                  42.2 / 27.6
//              8192 rows of 4, 512 x 512                    16.7 / 14.8
//              8192 rows of 1, 1024 x 768                   two 27.9, four 19.7
//   but        60 rows of 1, 1024 x 1024                    5.7 / 6.2
//              2 rows of 2, 4096 x 1024                     7.6 / 8.0
// No more units than clusters that run at once.  (K alone says when it is short, which is not
// best everywhere: 2 rows of 2, 1024 x 1024, would gain by two, 6.9 / 6.5.)
constexpr int kGroupMaxParts = 4;
int group_clusters(int log_parts);    // that the current device holds
inline int group_log_parts(long long units, long long K, int max_pairs) {
  if (K <= 8 * kGroupBK || 2 * units > max_pairs) return 0;
  if (4 * units <= max_pairs && units <= group_clusters(2)) return 2;
  return units <= group_clusters(1) ? 1 : 0;
}

// Clusters of `size` CTAs that the current device holds at once (152 SMs, one CTA on each: 36
// of 4, 15 of 8, since a cluster's CTAs share a GPC); asked once per device and kept in
// `known`.  0: not known.
template <typename... P>
int clusters_at_once(void (*kernel)(P...), unsigned size, int threads, int smem,
                     std::atomic<int> (&known)[64]) {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return 0;
  if ((n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim = {size, 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(size);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

struct GroupParams {
  int kind;
  int rows, groups;
  int first_group = 0;      // of those that offsets has; C and B are from it on
  // Products: C is rows x N, terms of the sums K.  Weights: C[g] is M x N (A's
  // columns x X's), the sums run over the group's rows (K == 0: without terms).
  int M, N, K;
  int tile_rows;            // most rows of a unit: 256, or 64 (products)
  int log_parts = 0;        // log2 of the pairs that share a unit's K: 1, or 2 or 4 where there
                            // are no more units than clusters
  int per_group;            // weights: tiles of a C[g]
  const int* offsets;       // null (groups 1): all rows are one group's
  int zmul;                 // 0: one B for all groups
  int seg;                  // k-tiles summed in tensor memory at a time
  float alpha, beta;
  void* C;
  long long ldc, stride_c;  // stride_c: weights
  unsigned* fault;
  unsigned long long timeout_ns;
};

// tmM: B as {K, N, groups} with boxes of 64 x 128 x 1 (forward), as {N, K,
// groups} with boxes of 64 x 128 x 1 (input), or X as {N, rows} with boxes of
// 64 x 64 (weights).  tmN, tmN16: X as {K, rows} with boxes of 64 x tile_rows / 2 and
// 64 x 16, or A as {M, rows} with boxes of 64 x 64 (weights; both alike).
cudaError_t launch_group(int dtype, int dtype_c, const GroupParams& p, const CUtensorMap* tmM,
                         const CUtensorMap* tmN, const CUtensorMap* tmN16, int pairs,
                         cudaStream_t stream);

}  // namespace dgemm
