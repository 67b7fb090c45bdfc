// C-ABI entry points of the grouped products: argument checks, tensor maps,
// operand copies and launch.  See include/dense_gemm_group.h.
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "group.h"
#include "group_operands.h"
#include "workspace.h"

namespace {

using namespace dgemm::api;

inline bool good_size(int n) { return n >= 0 && n <= GEMM_GROUP_MAX_SIZE; }
inline bool good_types(int dtype, int dtype_c) {
  return (dtype == 1 || dtype == 2) && (dtype_c == 0 || dtype_c == dtype);
}
}  // namespace

extern "C" {

gemm_status_t gemm_grouped(int dtype, gemm_op_t op_b, int dtype_c, int rows, int N, int K,
                           int groups, float alpha, const void* A, int lda, const void* B, int ldb,
                           long long stride_b, const int* offsets, float beta, void* C, int ldc,
                           cudaStream_t stream) {
  if (!good_types(dtype, dtype_c) || (op_b != GEMM_OP_N && op_b != GEMM_OP_T) ||
      !good_size(rows) || !good_size(N) || !good_size(K) || groups < 0 ||
      groups > GEMM_GROUP_MAX_GROUPS)
    return GEMM_ERR_INVALID_ARG;
  if (rows == 0 || N == 0 || groups == 0) return GEMM_OK;
  const int es = dtype_c == 0 ? 4 : 2;
  if (C == nullptr || ldc < N || offsets == nullptr) return GEMM_ERR_INVALID_ARG;
  if (!aligned(C, es) || !aligned(offsets, 4)) return GEMM_ERR_MISALIGNED;
  const uint64_t c_bytes = span(rows, (long long)N * es, (long long)ldc * es);
  if (overlap(C, c_bytes, offsets, (uint64_t)(groups + 1) * 4)) return GEMM_ERR_INVALID_ARG;
  const bool empty = K == 0 || alpha == 0.f;
  const bool t = op_b == GEMM_OP_T;
  Operand a{A, K, rows, lda, 1, 0, false};
  Operand b{B, t ? K : N, t ? N : K, ldb, groups, stride_b, false};
  gemm_status_t st;
  if (!empty) {
    if (stride_b < 0) return GEMM_ERR_INVALID_ARG;
    if ((st = a.check()) != GEMM_OK || (st = b.check()) != GEMM_OK) return st;
    if (overlap(C, c_bytes, A, a.bytes()) || overlap(C, c_bytes, B, b.bytes()))
      return GEMM_ERR_INVALID_ARG;
  } else if (beta == 1.f) {
    return GEMM_OK;
  }
  dgemm::GroupParams p;
  int max_pairs;
  if ((st = dgemm::current_device_pairs(&p.fault, &max_pairs)) != GEMM_OK) return st;
  dgemm::StreamWorkspaces workspaces(stream);   // held until everything is queued
  alignas(64) CUtensorMap tmM{}, tmN{}, tmN16{};
  p.tile_rows = dgemm::group_unit_rows(rows, groups);
  if (!empty) {
    if ((st = align_operands(a, b, workspaces, stream)) != GEMM_OK) return st;
    if (!encode_matrices(&tmM, dtype, b) || !encode_rows(&tmN, dtype, a, (uint32_t)p.tile_rows / 2) ||
        !encode_rows(&tmN16, dtype, a, 16))
      return GEMM_ERR_LAUNCH;
  }
  p.kind = t ? dgemm::kGroupForward : dgemm::kGroupInput;
  p.rows = rows, p.groups = groups;
  p.M = 0, p.N = N, p.K = empty ? 0 : K;
  p.per_group = 0;
  p.offsets = offsets;
  p.zmul = stride_b == 0 ? 0 : 1;
  p.seg = segment(dtype_c);
  p.alpha = empty ? 0.f : alpha, p.beta = beta;
  p.C = C, p.ldc = ldc, p.stride_c = 0;
  p.timeout_ns = dgemm::wait_bound_ns();
  const long long most = dgemm::group_units(rows, groups, N, p.tile_rows);
  p.log_parts = dgemm::group_log_parts(most, p.K, max_pairs);
  const long long want = most << p.log_parts;
  const int pairs = (int)(want < max_pairs ? want : max_pairs);
  return status_of(dgemm::launch_group(dtype, dtype_c, p, &tmM, &tmN, &tmN16, pairs, stream));
}

gemm_status_t gemm_grouped_grad(int dtype, int dtype_c, int rows, int M, int N, int groups,
                                float alpha, const void* A, int lda, const void* X, int ldx,
                                const int* offsets, float beta, void* C, int ldc,
                                long long stride_c, cudaStream_t stream) {
  if (!good_types(dtype, dtype_c) || !good_size(rows) || !good_size(M) || !good_size(N) ||
      groups < 0 || groups > GEMM_GROUP_MAX_GROUPS)
    return GEMM_ERR_INVALID_ARG;
  if (M == 0 || N == 0 || groups == 0) return GEMM_OK;
  const int es = dtype_c == 0 ? 4 : 2;
  const long long one = (long long)(M - 1) * ldc + N;   // elements that a C[g] spans
  if (C == nullptr || ldc < N || offsets == nullptr || (groups > 1 && stride_c < one))
    return GEMM_ERR_INVALID_ARG;
  if (!aligned(C, es) || !aligned(offsets, 4)) return GEMM_ERR_MISALIGNED;
  const uint64_t c_bytes = (uint64_t)((groups - 1) * (groups > 1 ? stride_c : 0) + one) * es;
  if (overlap(C, c_bytes, offsets, (uint64_t)(groups + 1) * 4)) return GEMM_ERR_INVALID_ARG;
  const bool empty = rows == 0 || alpha == 0.f;
  Operand a{A, M, rows, lda, 1, 0, false}, x{X, N, rows, ldx, 1, 0, false};
  gemm_status_t st;
  if (!empty) {
    if ((st = a.check()) != GEMM_OK || (st = x.check()) != GEMM_OK) return st;
    if (overlap(C, c_bytes, A, a.bytes()) || overlap(C, c_bytes, X, x.bytes()))
      return GEMM_ERR_INVALID_ARG;
  } else if (beta == 1.f) {
    return GEMM_OK;
  }
  dgemm::GroupParams p;
  int max_pairs;
  if ((st = dgemm::current_device_pairs(&p.fault, &max_pairs)) != GEMM_OK) return st;
  dgemm::StreamWorkspaces workspaces(stream);   // held until everything is queued
  alignas(64) CUtensorMap tmM{}, tmN{};
  if (!empty) {
    if ((st = align_operands(a, x, workspaces, stream)) != GEMM_OK) return st;
    if (!encode_rows(&tmM, dtype, x, 64) || !encode_rows(&tmN, dtype, a, 64))
      return GEMM_ERR_LAUNCH;
  }
  p.kind = dgemm::kGroupWeights;
  p.tile_rows = dgemm::kGroupTile;
  p.rows = rows, p.groups = groups;
  p.M = M, p.N = N, p.K = empty ? 0 : 1;
  p.per_group = ceil_div(M, dgemm::kGroupTile) * ceil_div(N, dgemm::kGroupTile);
  p.offsets = offsets;
  p.zmul = 0;
  p.seg = segment(dtype_c);
  p.alpha = empty ? 0.f : alpha, p.beta = beta;
  p.C = C, p.ldc = ldc, p.stride_c = groups > 1 ? stride_c : 0;
  p.timeout_ns = dgemm::wait_bound_ns();
  const long long units = (long long)groups * p.per_group;
  p.log_parts = dgemm::group_log_parts(units, empty ? 0 : rows / groups, max_pairs);
  const long long want = units << p.log_parts;
  const int pairs = (int)(want < max_pairs ? want : max_pairs);
  return status_of(dgemm::launch_group(dtype, dtype_c, p, &tmM, &tmN, &tmN, pairs, stream));
}

}  // extern "C"
