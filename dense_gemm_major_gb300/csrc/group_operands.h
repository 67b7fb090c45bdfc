// 16-bit operands of the grouped products and of those with 4-bit weights: checks,
// aligned copies, tensor maps.
#pragma once

#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "api_util.h"
#include "group.h"
#include "mx.h"
#include "workspace.h"

namespace dgemm {
namespace api {

inline CUtensorMapDataType map_type(int dtype) {
  return dtype == 1 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// A 16-bit operand: `count` matrices of `outer` rows of `inner` elements.
struct Operand {
  const void* p;
  long long inner, outer, ld, count, stride;
  bool packed;            // at any alignment: a copy with aligned rows is taken
  // The matrices lie behind one another (or are one, stride 0).
  gemm_status_t check() {
    if (p == nullptr || ld < inner) return GEMM_ERR_INVALID_ARG;
    const long long span1 = (outer - 1) * ld + inner;
    if (count > 1 && stride != 0 && stride < span1) return GEMM_ERR_INVALID_ARG;
    packed = false;
    if (aligned(p, 16) && ld % 8 == 0 && (count == 1 || stride % 8 == 0)) return GEMM_OK;
    packed = ld == inner && (count == 1 || stride == 0 || stride == outer * ld);
    return packed && aligned(p, 2) ? GEMM_OK : GEMM_ERR_MISALIGNED;
  }
  long long matrices() const { return stride == 0 ? 1 : count; }
  uint64_t bytes() const {
    return (uint64_t)((matrices() - 1) * stride + (outer - 1) * ld + inner) * 2;
  }
  long long copy_ld() const { return (inner + 7) / 8 * 8; }
  size_t copy_bytes() const {   // a multiple of 256
    return packed ? ((size_t)(matrices() * outer * copy_ld()) * 2 + 255) / 256 * 256 : 0;
  }
  gemm_status_t copy_to(void* to, cudaStream_t stream) {
    const long long ldd = copy_ld();
    const gemm_status_t st = status_of(
        launch_mx_align(p, matrices() * outer, (int)inner, to, ldd, stream));
    p = to;
    ld = ldd;
    stride = stride == 0 ? 0 : outer * ldd;
    return st;
  }
};

// Operands that TMA cannot address become copies in the workspace that `ws` holds.
inline gemm_status_t align_operands(Operand& a, Operand& b, StreamWorkspaces& ws,
                             cudaStream_t stream) {
  if (!a.packed && !b.packed) return GEMM_OK;
  void* p = nullptr;
  gemm_status_t st = ws.get(kWsPack, a.copy_bytes() + b.copy_bytes(), &p);
  if (st != GEMM_OK) return st;
  char* const second = static_cast<char*>(p) + a.copy_bytes();
  if (a.packed && (st = a.copy_to(p, stream)) != GEMM_OK) return st;
  if (b.packed && (st = b.copy_to(second, stream)) != GEMM_OK) return st;
  return GEMM_OK;
}

inline bool encode_rows(CUtensorMap* map, int dtype, const Operand& o, uint32_t box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)o.inner, (cuuint64_t)o.outer};
  const cuuint64_t strides[1] = {(cuuint64_t)o.ld * 2};
  const cuuint32_t box[2] = {64, box_rows};
  return encode_tiled(map, map_type(dtype), 2, o.p, dims, strides, box);
}
inline bool encode_matrices(CUtensorMap* map, int dtype, const Operand& o) {
  const cuuint64_t dims[3] = {(cuuint64_t)o.inner, (cuuint64_t)o.outer,
                              (cuuint64_t)o.matrices()};
  // (The distance of a single matrix's successor: never used, but checked.)
  const cuuint64_t far = (cuuint64_t)(o.stride != 0 && o.count > 1 ? o.stride : o.outer * o.ld);
  const cuuint64_t strides[2] = {(cuuint64_t)o.ld * 2, far * 2};
  const cuuint32_t box[3] = {64, 128, 1};
  return encode_tiled(map, map_type(dtype), 3, o.p, dims, strides, box);
}

// k-tiles per sum in tensor memory, which truncates at each step of 16: sums of
// like terms come out too small, the more the longer they are.  FP32 results:
// 1024 terms, 16-bit ones 16384 (a fifth of FP16's rounding).
inline int segment(int dtype_c) { return (dtype_c == 0 ? 1024 : 16384) / kGroupBK; }

}  // namespace api
}  // namespace dgemm
