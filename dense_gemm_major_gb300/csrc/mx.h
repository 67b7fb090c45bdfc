// Internal interface of the microscaled (MX) operators: the kernels' launch
// functions, called by mx_api.cu.  Callers use include/dense_gemm_mx.h.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "dense_gemm_mx.h"
#include "launch.h"

namespace dgemm {

constexpr int kMxBlock = 32;         // values that share a scale
constexpr int kMxTileRows = 128;     // a tile of scales: 128 rows x 4 blocks,
constexpr int kMxTileBlocks = 4;     //   512 bytes
constexpr int kMxTileBytes = 512;

__host__ __device__ inline int mx_blocks(int K) { return (K + kMxBlock - 1) / kMxBlock; }
// Tiles of scales along a row of K columns.
__host__ __device__ inline int mx_scale_tiles(int K) {
  return (mx_blocks(K) + kMxTileBlocks - 1) / kMxTileBlocks;
}

// Quantisation; the arguments of gemm_mx_quantize, checked.
cudaError_t launch_mx_quantize(int fmt, int dtype, int op, int R, int K, const void* X,
                               long long ldx, void* codes, long long ldq, void* scales,
                               cudaStream_t stream);
cudaError_t launch_mx_dequantize(int fmt, int dtype, int R, int K, const void* codes,
                                 long long ldq, const void* scales, void* Y, long long ldy,
                                 cudaStream_t stream);

// C := alpha * A . B^T + beta * C on tcgen05 block-scaled FP4.  The kernel
// puts B's rows (C's columns) on the MMA's M side, so that a warp's 32 TMEM
// lanes are 32 consecutive columns of a row of C.
struct Mx4Params {
  int M, N, K;                        // C is M x N
  const unsigned char* sa;            // scales of A and B
  const unsigned char* sb;
  int tiles_m, tiles_n;               // tiles of C
  int group;                          // tile columns of C per rasterisation group
  float alpha, beta;
  void* C;
  long long ldc;
  int dtype;                          // of C
  unsigned* fault;
  unsigned long long timeout_ns;
};
constexpr int kMx4BN = 128;           // rows of B (columns of C) per tile
constexpr int kMx4BM = 128;           // rows of A (rows of C) per tile
constexpr int kMx4BK = 256;           // 128 bytes of codes
cudaError_t launch_mx4(const Mx4Params& p, const CUtensorMap* tmA, const CUtensorMap* tmB,
                       int grid, cudaStream_t stream);

// C := alpha * op(A) . B + beta * C, B quantised (K x N).
struct MxGradParams {
  int M, N, K;
  int fmt, dtype, op_a, dtype_c;
  const unsigned char* codes;
  long long ldb;
  const unsigned char* sb;
  int tiles_m, tiles_n;
  int group;
  float alpha, beta;
  void* C;
  long long ldc;
  unsigned* fault;
  unsigned long long timeout_ns;
};
constexpr int kMxGradBN = 128;        // columns of B (and C) per tile: the MMA's M side
constexpr int kMxGradBM = 256;        // rows of C per tile: the MMA's N side
constexpr int kMxGradBK = 64;
cudaError_t launch_mx_grad(const MxGradParams& p, const CUtensorMap* tmA, int grid,
                           cudaStream_t stream);

}  // namespace dgemm
