// Internal interface of the microscaled (MX) operators: the kernels' launch
// functions, called by mx_api.cu.  Callers use include/dense_gemm_mx.h.
#pragma once

#include <atomic>
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

// Dynamic shared memory of `kernel`, allowed once per device: `done` (a static
// of the caller) has a bit per device.
template <typename... Params>
cudaError_t mx_allow_smem(void (*kernel)(Params...), int bytes, std::atomic<uint64_t>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit & done->load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// The current device's fault word, and the CTA pairs that it can hold at once
// with one CTA per SM (fewer than half of its SMs: a cluster's CTAs share a
// GPC; a pair too many would run after all others).  In api.cu.
gemm_status_t current_device_pairs(unsigned** fault, int* pairs);

// Quantisation; the arguments of gemm_mx_quantize, checked.
cudaError_t launch_mx_quantize(int fmt, int dtype, int op, int R, int K, const void* X,
                               long long ldx, void* codes, long long ldq, void* scales,
                               cudaStream_t stream);
cudaError_t launch_mx_dequantize(int fmt, int dtype, int R, int K, const void* codes,
                                 long long ldq, const void* scales, void* Y, long long ldy,
                                 cudaStream_t stream);

// Schedule of the kernels that compute 256 x 256 tiles of C on CTA pairs:
// tiles [0, full_tiles) whole and the rest as two halves of 128 rows of C
// (by_halves: all of C as halves), each over `slices` ranges of K (slices > 1:
// FP32 partial results at ws + slice * M * ldw, summed by launch_mx_reduce).
struct MxSchedule {
  int tiles_m, tiles_n;     // tiles of C along its rows and columns
  int halves_m;             // halves along its rows
  int by_halves;
  int full_tiles, units;    // units: all halves and tiles, times slices
  int slices;
  int group;                // tile columns per rasterisation group
};
constexpr int kMxPairTile = 256;

// D (16-byte aligned rows of ldd elements, a multiple of 8) := S, rows x cols
// packed 16-bit elements.
cudaError_t launch_mx_align(const void* S, long long rows, int cols, void* D, long long ldd,
                            cudaStream_t stream);

// C := alpha * (the sum over s of ws[s * M * ldw + i * ldw + j], in slice
// order) + beta * C; dtype of C.  ldw is a multiple of 4.
cudaError_t launch_mx_reduce(const float* ws, int slices, int M, int N, long long ldw, float alpha,
                             float beta, void* C, long long ldc, int dtype, cudaStream_t stream);

// C := alpha * A . B^T + beta * C on tcgen05 block-scaled FP4.
struct Mx4Params {
  int M, N, K;                        // C is M x N
  MxSchedule sched;
  float* ws;
  long long ldw;
  float alpha, beta;
  void* C;
  long long ldc;
  int dtype;                          // of C
  unsigned* fault;
  unsigned long long timeout_ns;
};
constexpr int kMx4BK = 512;
// Terms of an FP32 result that the 4-bit products sum in tensor memory at a time.
constexpr int kMx4SegTerms = 4096;
// tmA, tmB: codes as bytes, boxes of 128 bytes x 64 and 128 rows; tmSA, tmSB:
// scales as 64-bit words, one row per 128 rows of the operand, boxes of four
// tiles.
cudaError_t launch_mx4(const Mx4Params& p, const CUtensorMap* tmA, const CUtensorMap* tmB,
                       const CUtensorMap* tmSA, const CUtensorMap* tmSB, int pairs,
                       cudaStream_t stream);

// C := alpha * A . B^T + beta * C for up to 64 rows of A, which are given in
// MXFP4 (tmA, sa) or, up to 48, as an array X of dtype that the kernel
// quantises.
struct Mx4FewParams {
  int M, N, K;
  const void* X;              // null: A in MXFP4
  long long ldx;
  bool vec;                   // rows of X are 16-byte aligned
  const unsigned char* sa;    // scales of A and B
  const unsigned char* sb;
  int split;                  // CTAs (a cluster) that share a tile's K
  float alpha, beta;
  void* C;
  long long ldc;
  int dtype;                  // of C (and X)
  unsigned* fault;
  unsigned long long timeout_ns;
};
// The pair kernel against this one at 64 rows, N x K, us: 512 x 512 4.6 / 4.4, 1024
// x 1024 5.0 / 4.1, 2048 x 8192 9.2 / 7.4, 8192 x 8192 11.7 / 8.3, 4096 x 14336
// 11.3 / 9.8, 65536 x 2048 14.9 / 14.2, but 2048 x 2048 5.8 / 6.4, 4096 x 4096 7.3 /
// 7.8, 8192 x 1024 5.2 / 5.9, 16384 x 4096 8.2 / 8.5: short rows leave the cluster
// little to share, and tiles of 256 columns few rounds.  At 56 rows those are 5.8 / 5.9, 7.3 / 7.2, 5.2 / 5.7 and 9.0 /
// 8.3; at 32 this one is quicker in all.  (With a tile of 128 rows the pairs
// were: 128 x 2048 x 2048 7.7 / 9.7 us.)
constexpr int kMx4FewRows = 64, kMx4FewBK = 256;
inline int mx4_few_rows(int N, int K) {
  return N >= 2048 && N <= 16384 && K <= 4096 ? kMx4FewRows - 8 : kMx4FewRows;
}
// Quantising A inside the kernel saves a launch (1.2 us of the GPU and 2.7 us
// of a calling thread), but each CTA then quantises the rows' part that it
// multiplies: M times its share of K values, done anew for every 128 columns.
// Where the CTAs run in several waves that counts for each.  Inside / before, us,
// up to 16 rows: 16384 values 1024 x 8192 (N x K), 16 rows 4.9 / 5.8, 4096 x 4096,
// 16 rows (8192) 5.7 / 6.7, 16384 x 4096, 8 rows 7.4 / 8.4; 28672 values 4096 x
// 14336, 16 rows 8.6 / 8.6; 32768 values 16384 x 4096, 16 rows 8.4 / 8.1, 65536 x
// 2048, 8 rows (two waves) 12.4 / 11.7.  With more rows a stage's blocks are
// three passes of its warps' lanes or more, which pays for one or two stages:
// 4096 x 4096 (two), 17 / 24 / 33 / 48 rows 7.0 / 6.9 / 7.8 / 9.0 and 7.0 / 7.4 /
// 8.0 / 8.8, 2048 x 2048 (one), 24 / 40 rows 5.4 / 6.5 and 6.0 / 6.8; but 1024 x
// 8192 (four), 17 / 24 rows 7.2 / 6.5 and 6.2 / 6.3, 2048 x 8192 8.0 / 7.6 and
// 7.0 / 7.1.
constexpr int kMx4FewRawRows = 48, kMx4FewRawValues = 24 * 1024;
constexpr int kMx4FewRawShort = 16, kMx4FewRawStages = 2;
// Rows of A that the kernel computes for M of them.
inline int mx4_few_tile(int M) { return M <= 16 ? 16 : (M <= 32 ? 32 : 64); }
// tmA: A's codes as bytes, boxes of 128 bytes x mx4_few_tile(M) rows; tmB:
// B's, boxes of 128 bytes x 128 rows.
cudaError_t launch_mx4_few(const Mx4FewParams& p, const CUtensorMap* tmA, const CUtensorMap* tmB,
                           cudaStream_t stream);

// C := alpha * op(A) . B + beta * C, B quantised (K x N).
struct MxGradParams {
  int M, N, K;
  int fmt, dtype, op_a, dtype_c;
  const unsigned char* sb;
  MxSchedule sched;
  int seg;                  // k-tiles summed in tensor memory at a time
  float* ws;
  long long ldw;
  float alpha, beta;
  void* C;
  long long ldc;
  unsigned* fault;
  unsigned long long timeout_ns;
};
constexpr int kMxGradBK = 128;
// tmA: op(A), boxes of 64 x 64; tmB: the codes as bytes, boxes of 128 rows x
// 128 columns.
cudaError_t launch_mx_grad(const MxGradParams& p, const CUtensorMap* tmA, const CUtensorMap* tmB,
                           int pairs, cudaStream_t stream);

}  // namespace dgemm
