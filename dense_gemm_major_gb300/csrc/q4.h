// Internal interface of the products with 4-bit weights and group scales: the
// kernels' launch functions, called by q4_api.cu.  Callers use
// include/dense_gemm_q4.h.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "dense_gemm_q4.h"
#include "launch.h"

namespace dgemm {

// Few rows: a CTA computes 64 columns of Y (rows of W) for 8 or 16 rows of one expert, over
// its share of K or one after the other.
constexpr int kQ4TileN = 64;
constexpr int kQ4BK = 512;
// Groups of columns of a row (K > 0).  (Not from K + group - 1, which for a large group is
// past what an int holds.)
__host__ __device__ inline int q4_groups(int K, int group) { return (K - 1) / group + 1; }

struct Q4FewParams {
  int rows, N, K, group;
  int experts;              // 0: one matrix for all rows
  const int* offsets;
  int tile_rows;            // rows of Y per CTA
  int slots;                // upper bound of tiles of rows
  int split;                // CTAs (a cluster) that share a tile's K
  int max_ctas;             // as many as run at once
  const void* scales;
  const unsigned char* zeros;
  void* Y;
  long long ldy;
  unsigned* fault;
  unsigned long long timeout_ns;
};
// tmQ: the codes as bytes {ceil(K / 2), N, experts} with boxes of 128 x 64 x 1; tmX: X
// as {K, rows} with boxes of 64 x tile_rows.
cudaError_t launch_q4_few(int dtype, const Q4FewParams& p, const CUtensorMap* tmQ,
                          const CUtensorMap* tmX, cudaStream_t stream);

// Clusters of `split` (up to 8) CTAs that the current device holds at once.
int q4_few_clusters(int split);
int q4_rows_clusters(int split);

// More rows: 128 columns of Y for up to 128 rows of one expert, over a share of K or one after
// the other.
constexpr int kQ4RowsTileN = 128;
constexpr int kQ4RowsBK = 128;
inline int q4_rows_tile(int rows) {
  return rows <= 16 ? 16 : (rows <= 32 ? 32 : (rows <= 64 ? 64 : 128));
}
// tmQ: the codes with boxes of 128 x 128 x 1; tmX: boxes of 64 x tile_rows.
cudaError_t launch_q4_rows(int dtype, const Q4FewParams& p, const CUtensorMap* tmQ,
                           const CUtensorMap* tmX, cudaStream_t stream);

// D (experts x N rows of K values of dtype, pitch ldd, a multiple of 8) := the
// weights of `experts` matrices, or N rows of them: their codes stride_q bytes apart,
// their scales and zeros scale_n to a group.  Experts without rows by `offsets`
// (null: one without) are left out.
cudaError_t launch_q4_values(int dtype, int group, int experts, int N, int K, int scale_n,
                             const unsigned char* codes, int ldq, long long stride_q,
                             const void* scales, const unsigned char* zeros, const int* offsets,
                             void* D, long long ldd, cudaStream_t stream);

}  // namespace dgemm
