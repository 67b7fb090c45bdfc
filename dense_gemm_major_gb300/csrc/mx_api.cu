// C-ABI entry points of the microscaled (MX) operators: argument checks,
// tensor maps, workspaces and launch.  See include/dense_gemm_mx.h.
#include <cstdint>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "dense_gemm_mx.h"
#include "launch.h"
#include "mx.h"
#include "workspace.h"

namespace {

// cuTensorMapEncodeTiled, fetched from the driver once.
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// 2-D row-major array {inner, outer}.
bool encode_2d(CUtensorMap* map, CUtensorMapDataType dt, const void* base, uint64_t inner,
               uint64_t outer, uint64_t pitch_bytes, uint32_t box_inner, uint32_t box_outer,
               bool swizzle = true) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {pitch_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, dt, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline bool aligned(const void* p, int n) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(n - 1)) == 0;
}
inline int ceil_div(int a, int b) { return (a + b - 1) / b; }
inline int elem_size(int dtype) { return dtype == 0 ? 4 : 2; }
inline bool good_format(int fmt) { return fmt == GEMM_MXFP4 || fmt == GEMM_MXINT8; }
inline bool good_dtype(int d) { return d >= 0 && d <= 2; }
inline bool good_size(int n) { return n >= 0 && n <= GEMM_MX_MAX_SIZE; }
inline bool good_op(int op) { return op == GEMM_OP_N || op == GEMM_OP_T; }

inline uint64_t span(long long rows, long long width, long long pitch) {
  return rows > 0 && width > 0 ? (uint64_t)((rows - 1) * pitch + width) : 0;
}
inline bool overlap(const void* a, uint64_t an, const void* b, uint64_t bn) {
  if (an == 0 || bn == 0 || a == nullptr || b == nullptr) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + bn && b0 < a0 + an;
}

inline int code_bytes(int fmt, int K) { return fmt == GEMM_MXFP4 ? K / 2 + (K & 1) : K; }
inline int code_ld(int fmt, int K) {
  return (int)(((long long)code_bytes(fmt, K) + 15) / 16 * 16);
}
inline long long scale_bytes(int R, int K) {
  return (long long)((R + 127ll) / 128) * dgemm::mx_scale_tiles(K) * dgemm::kMxTileBytes;
}

// A quantised R x K operand (R, K > 0) that a kernel reads or writes.
gemm_status_t check_quantized(int fmt, int K, const void* codes, int ldq, const void* scales) {
  if (codes == nullptr || scales == nullptr || ldq < code_ld(fmt, K)) return GEMM_ERR_INVALID_ARG;
  if (!aligned(codes, 16) || !aligned(scales, 16) || ldq % 16 != 0) return GEMM_ERR_MISALIGNED;
  return GEMM_OK;
}
inline bool overlaps_quantized(const void* p, uint64_t n, int fmt, int R, int K,
                               const void* codes, int ldq, const void* scales) {
  return overlap(p, n, codes, span(R, code_bytes(fmt, K), ldq)) ||
         overlap(p, n, scales, (uint64_t)scale_bytes(R, K));
}

gemm_status_t status_of(cudaError_t e) {
  if (e == cudaSuccess) return GEMM_OK;
  cudaGetLastError();
  return GEMM_ERR_LAUNCH;
}

// C := beta * C, the product with no terms.
gemm_status_t scale_only(int dtype, int M, int N, float beta, void* C, int ldc,
                         cudaStream_t stream) {
  if (beta == 1.f) return GEMM_OK;
  return status_of(dgemm::launch_scale_c(C, M, N, ldc, dtype, beta, stream));
}

// Schedule of an M x N product of nk k-tiles on `pairs` CTA pairs: whole
// 256 x 256 tiles (those of a last partial round as halves, when the halves
// fit one round), or halves of 128 rows, each over 1 .. kMaxSlices ranges of
// K; whichever the model below, in us, finds quickest.  Its constants are
// measured on GB300 (per kernel: a k-tile of a whole tile and of a half; the
// rest is common).
struct StageCost {
  double whole, half;
};
constexpr int kMaxSlices = 16;
constexpr long long kWorkspaceCap = 256ll << 20;   // bytes of partial results
constexpr double kUnitCost = 1.2;                  // pipeline fill, drain, store
constexpr double kReduceCost = 2.0;                // the launch that sums the slices,
constexpr double kReduceBytesPerUs = 3e6;          // and what is written and read for it
dgemm::MxSchedule schedule(int M, int N, int nk, int pairs, int group, StageCost cost) {
  dgemm::MxSchedule sc;
  sc.tiles_m = ceil_div(M, dgemm::kMxPairTile);
  sc.tiles_n = ceil_div(N, dgemm::kMxPairTile);
  sc.halves_m = ceil_div(M, dgemm::kMxPairTile / 2);
  sc.group = group;
  const long long tiles = (long long)sc.tiles_m * sc.tiles_n;
  const long long halves = (long long)sc.halves_m * sc.tiles_n;
  const long long slice_bytes = (long long)M * (((long long)N + 3) / 4 * 4) * 4;
  double best = -1.0;
  auto take = [&](double us, bool by_halves, int slices) {
    if (best >= 0.0 && us >= best - 1e-9) return;
    best = us;
    sc.by_halves = by_halves ? 1 : 0;
    sc.slices = slices;
  };
  for (int s = 1; s <= kMaxSlices && s <= nk; ++s) {
    if (s > 1 && s * slice_bytes > kWorkspaceCap) break;
    const double k = (double)ceil_div(nk, s);
    const double extra = s > 1 ? kReduceCost + (double)(s * slice_bytes) / kReduceBytesPerUs : 0.0;
    const long long hr = (halves * s + pairs - 1) / pairs;
    take((double)hr * (k * cost.half + kUnitCost) + extra, true, s);
    const long long rem = tiles * s % pairs;
    const bool split_rest = s == 1 && rem > 0 && 2 * rem <= pairs;
    double us = (double)(tiles * s / pairs) * (k * cost.whole + kUnitCost);
    if (rem > 0) us += (split_rest ? k * cost.half : k * cost.whole) + kUnitCost;
    take(us + extra, false, s);
  }
  if (sc.by_halves) {
    sc.full_tiles = 0;
    sc.units = (int)(halves * sc.slices);
  } else {
    const long long rem = tiles % pairs;
    sc.full_tiles = (int)(sc.slices == 1 && 2 * rem <= pairs ? tiles - rem : tiles);
    sc.units = (int)((sc.full_tiles + 2 * (tiles - sc.full_tiles)) * sc.slices);
  }
  return sc;
}

// The workspace of a schedule with slices.
gemm_status_t partials(const dgemm::MxSchedule& sc, int M, int N,
                       dgemm::StreamWorkspaces& workspaces, float** ws, long long* ldw) {
  *ws = nullptr;
  *ldw = ((long long)N + 3) / 4 * 4;
  if (sc.slices == 1) return GEMM_OK;
  void* p = nullptr;
  const gemm_status_t st =
      workspaces.get(dgemm::kWsPartials, (size_t)sc.slices * M * *ldw * 4, &p);
  *ws = static_cast<float*>(p);
  return st;
}

// CTAs of the few-row kernel that share a tile's K: as many (2, 4 or 8 of a
// cluster) as keep one wave of two CTAs per SM, each with a stage at least.
int few_split(int N, int K, int max_pairs) {
  const int tiles = ceil_div(N, 128), nk = ceil_div(K, dgemm::kMx4FewBK);
  int split = 1;
  while (split < 8 && 2 * split <= nk && 2 * split * tiles <= 4 * max_pairs) split *= 2;
  return split;
}

// Whether the few-row kernel quantises A itself: see kMx4FewRawRows.
bool few_raw(int M, int N, int K, int max_pairs) {
  const int split = few_split(N, K, max_pairs);
  const long long waves = ((long long)ceil_div(N, 128) * split + 4 * max_pairs - 1) / (4 * max_pairs);
  const long long stages = ceil_div(ceil_div(K, dgemm::kMx4FewBK), split) * waves;
  return M <= dgemm::kMx4FewRawRows &&
         M * stages * dgemm::kMx4FewBK <= dgemm::kMx4FewRawValues &&
         (M <= dgemm::kMx4FewRawShort || stages <= dgemm::kMx4FewRawStages);
}

// The product of checked operands, 0 < M <= mx4_few_rows(), N, K > 0; A is X,
// unquantised, or a.
gemm_status_t run_few(int dtype, int M, int N, int K, float alpha, const void* X, long long ldx,
                      const void* a, long long lda, const void* sa, const void* b, long long ldb,
                      const void* sb, float beta, void* C, int ldc, unsigned* fault,
                      int max_pairs, cudaStream_t stream) {
  alignas(64) CUtensorMap tmA{}, tmB;
  const uint64_t width = (uint64_t)code_bytes(GEMM_MXFP4, K);
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  if (!encode_2d(&tmB, u8, b, width, (uint64_t)N, (uint64_t)ldb, 128, 128) ||
      (X == nullptr && !encode_2d(&tmA, u8, a, width, (uint64_t)M, (uint64_t)lda, 128,
                                  (uint32_t)dgemm::mx4_few_tile(M))))
    return GEMM_ERR_LAUNCH;
  dgemm::Mx4FewParams p;
  p.M = M, p.N = N, p.K = K;
  p.X = X, p.ldx = ldx;
  p.vec = aligned(X, 16) && (ldx * elem_size(dtype)) % 16 == 0;
  p.sa = static_cast<const unsigned char*>(sa);
  p.sb = static_cast<const unsigned char*>(sb);
  p.split = few_split(N, K, max_pairs);
  p.alpha = alpha, p.beta = beta;
  p.C = C, p.ldc = ldc, p.dtype = dtype;
  p.fault = fault, p.timeout_ns = dgemm::wait_bound_ns();
  return status_of(dgemm::launch_mx4_few(p, &tmA, &tmB, stream));
}

// The product of checked operands, M, N, K > 0.
gemm_status_t run_mx4(int dtype, int M, int N, int K, float alpha, const void* a, long long lda,
                      const void* sa, const void* b, long long ldb, const void* sb, float beta,
                      void* C, int ldc, unsigned* fault, int max_pairs,
                      dgemm::StreamWorkspaces& workspaces, cudaStream_t stream) {
  if (M <= dgemm::mx4_few_rows(N, K))
    return run_few(dtype, M, N, K, alpha, nullptr, 0, a, lda, sa, b, ldb, sb, beta, C, ldc, fault,
                   max_pairs, stream);
  alignas(64) CUtensorMap tmA, tmB, tmSA, tmSB;
  const uint64_t width = (uint64_t)code_bytes(GEMM_MXFP4, K);
  const uint64_t srow = (uint64_t)dgemm::mx_scale_tiles(K) * dgemm::kMxTileBytes;
  constexpr uint32_t sbox = dgemm::kMx4BK / 128 * dgemm::kMxTileBytes / 8;
  const CUtensorMapDataType u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const CUtensorMapDataType u64 = CU_TENSOR_MAP_DATA_TYPE_UINT64;
  if (!encode_2d(&tmA, u8, a, width, (uint64_t)M, (uint64_t)lda, 128, 64) ||
      !encode_2d(&tmB, u8, b, width, (uint64_t)N, (uint64_t)ldb, 128, 128) ||
      !encode_2d(&tmSA, u64, sa, srow / 8, (uint64_t)ceil_div(M, 128), srow, sbox, 1, false) ||
      !encode_2d(&tmSB, u64, sb, srow / 8, (uint64_t)ceil_div(N, 128), srow, sbox, 1, false))
    return GEMM_ERR_LAUNCH;
  dgemm::Mx4Params p;
  p.M = M, p.N = N, p.K = K;
  // (Groups of 2 / 8 / 64 tile columns: 8192^3 150 / 156 / 152 us, but 16384^3,
  // whose operands L2 does not hold, 1199 / 1095 / 1330.)
  p.sched = schedule(M, N, ceil_div(K, dgemm::kMx4BK), max_pairs, 8, {0.70, 0.44});
  gemm_status_t st = partials(p.sched, M, N, workspaces, &p.ws, &p.ldw);
  if (st != GEMM_OK) return st;
  p.alpha = alpha, p.beta = beta;
  p.C = C, p.ldc = ldc, p.dtype = dtype;
  p.fault = fault, p.timeout_ns = dgemm::wait_bound_ns();
  const int pairs = p.sched.units < max_pairs ? p.sched.units : max_pairs;
  cudaError_t e = dgemm::launch_mx4(p, &tmA, &tmB, &tmSA, &tmSB, pairs, stream);
  if (e == cudaSuccess && p.sched.slices > 1)
    e = dgemm::launch_mx_reduce(p.ws, p.sched.slices, M, N, p.ldw, alpha, beta, C, ldc, dtype,
                                stream);
  return status_of(e);
}

}  // namespace

extern "C" {

int gemm_mx_code_ld(gemm_mx_format_t fmt, int K) {
  if (!good_format(fmt) || !good_size(K)) return -1;
  return code_ld(fmt, K);
}

long long gemm_mx_scale_bytes(int R, int K) {
  if (!good_size(R) || !good_size(K)) return -1;
  return scale_bytes(R, K);
}

gemm_status_t gemm_mx_quantize(gemm_mx_format_t fmt, int dtype, gemm_op_t op, int R, int K,
                               const void* X, int ldx, void* codes, int ldq, void* scales,
                               cudaStream_t stream) {
  if (!good_format(fmt) || !good_dtype(dtype) || !good_op(op) || !good_size(R) ||
      !good_size(K))
    return GEMM_ERR_INVALID_ARG;
  if (R == 0 || K == 0) return GEMM_OK;
  const int es = elem_size(dtype);
  if (X == nullptr || ldx < (op == GEMM_OP_N ? K : R)) return GEMM_ERR_INVALID_ARG;
  gemm_status_t st = check_quantized(fmt, K, codes, ldq, scales);
  if (st != GEMM_OK) return st;
  if (!aligned(X, es)) return GEMM_ERR_MISALIGNED;
  const uint64_t xs = op == GEMM_OP_N ? span(R, (long long)K * es, (long long)ldx * es)
                                      : span(K, (long long)R * es, (long long)ldx * es);
  if (overlaps_quantized(X, xs, fmt, R, K, codes, ldq, scales) ||
      overlap(codes, span(R, code_bytes(fmt, K), ldq), scales, (uint64_t)scale_bytes(R, K)))
    return GEMM_ERR_INVALID_ARG;
  unsigned* fault;
  int max_pairs;
  if ((st = dgemm::current_device_pairs(&fault, &max_pairs)) != GEMM_OK) return st;
  return status_of(
      dgemm::launch_mx_quantize(fmt, dtype, op, R, K, X, ldx, codes, ldq, scales, stream));
}

gemm_status_t gemm_mx_dequantize(gemm_mx_format_t fmt, int dtype, int R, int K,
                                 const void* codes, int ldq, const void* scales, void* Y, int ldy,
                                 cudaStream_t stream) {
  if (!good_format(fmt) || !good_dtype(dtype) || !good_size(R) || !good_size(K))
    return GEMM_ERR_INVALID_ARG;
  if (R == 0 || K == 0) return GEMM_OK;
  const int es = elem_size(dtype);
  if (Y == nullptr || ldy < K) return GEMM_ERR_INVALID_ARG;
  gemm_status_t st = check_quantized(fmt, K, codes, ldq, scales);
  if (st != GEMM_OK) return st;
  if (!aligned(Y, es)) return GEMM_ERR_MISALIGNED;
  if (overlaps_quantized(Y, span(R, (long long)K * es, (long long)ldy * es), fmt, R, K, codes,
                         ldq, scales))
    return GEMM_ERR_INVALID_ARG;
  unsigned* fault;
  int max_pairs;
  if ((st = dgemm::current_device_pairs(&fault, &max_pairs)) != GEMM_OK) return st;
  return status_of(
      dgemm::launch_mx_dequantize(fmt, dtype, R, K, codes, ldq, scales, Y, ldy, stream));
}

gemm_status_t gemm_mx4(int dtype, int M, int N, int K, float alpha, const void* a_codes, int lda,
                       const void* a_scales, const void* b_codes, int ldb, const void* b_scales,
                       float beta, void* C, int ldc, cudaStream_t stream) {
  if (!good_dtype(dtype) || !good_size(M) || !good_size(N) || !good_size(K))
    return GEMM_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return GEMM_OK;
  const int es = elem_size(dtype);
  if (C == nullptr || ldc < N) return GEMM_ERR_INVALID_ARG;
  if (!aligned(C, es)) return GEMM_ERR_MISALIGNED;
  const bool empty = K == 0 || alpha == 0.f;
  gemm_status_t st;
  if (!empty) {
    const uint64_t cs = span(M, (long long)N * es, (long long)ldc * es);
    if ((st = check_quantized(GEMM_MXFP4, K, a_codes, lda, a_scales)) != GEMM_OK ||
        (st = check_quantized(GEMM_MXFP4, K, b_codes, ldb, b_scales)) != GEMM_OK)
      return st;
    if (overlaps_quantized(C, cs, GEMM_MXFP4, M, K, a_codes, lda, a_scales) ||
        overlaps_quantized(C, cs, GEMM_MXFP4, N, K, b_codes, ldb, b_scales))
      return GEMM_ERR_INVALID_ARG;
  }
  unsigned* fault;
  int max_pairs;
  if ((st = dgemm::current_device_pairs(&fault, &max_pairs)) != GEMM_OK) return st;
  if (empty) return scale_only(dtype, M, N, beta, C, ldc, stream);
  dgemm::StreamWorkspaces workspaces(stream);
  return run_mx4(dtype, M, N, K, alpha, a_codes, lda, a_scales, b_codes, ldb, b_scales, beta, C,
                 ldc, fault, max_pairs, workspaces, stream);
}

gemm_status_t gemm_mx4_linear(int dtype, int M, int N, int K, const void* X, int ldx,
                              const void* w_codes, int ldw, const void* w_scales, void* Y,
                              int ldy, cudaStream_t stream) {
  if (!good_dtype(dtype) || !good_size(M) || !good_size(N) || !good_size(K))
    return GEMM_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return GEMM_OK;
  const int es = elem_size(dtype);
  if (Y == nullptr || ldy < N) return GEMM_ERR_INVALID_ARG;
  if (!aligned(Y, es)) return GEMM_ERR_MISALIGNED;
  gemm_status_t st;
  if (K > 0) {
    if (X == nullptr || ldx < K) return GEMM_ERR_INVALID_ARG;
    if ((st = check_quantized(GEMM_MXFP4, K, w_codes, ldw, w_scales)) != GEMM_OK) return st;
    if (!aligned(X, es)) return GEMM_ERR_MISALIGNED;
    const uint64_t ys = span(M, (long long)N * es, (long long)ldy * es);
    if (overlap(Y, ys, X, span(M, (long long)K * es, (long long)ldx * es)) ||
        overlaps_quantized(Y, ys, GEMM_MXFP4, N, K, w_codes, ldw, w_scales))
      return GEMM_ERR_INVALID_ARG;
  }
  unsigned* fault;
  int max_pairs;
  if ((st = dgemm::current_device_pairs(&fault, &max_pairs)) != GEMM_OK) return st;
  if (K == 0) return scale_only(dtype, M, N, 0.f, Y, ldy, stream);
  if (few_raw(M, N, K, max_pairs))
    return run_few(dtype, M, N, K, 1.f, X, ldx, nullptr, 0, nullptr, w_codes, ldw, w_scales, 0.f,
                   Y, ldy, fault, max_pairs, stream);
  const int ldq = code_ld(GEMM_MXFP4, K);
  const size_t code_size = ((size_t)M * ldq + 255) / 256 * 256;
  dgemm::StreamWorkspaces workspaces(stream);   // held until the product is queued
  void* p = nullptr;
  st = workspaces.get(dgemm::kWsQuantized, code_size + (size_t)scale_bytes(M, K), &p);
  if (st != GEMM_OK) return st;
  unsigned char* const ws = static_cast<unsigned char*>(p);
  st = status_of(dgemm::launch_mx_quantize(GEMM_MXFP4, dtype, GEMM_OP_N, M, K, X, ldx, ws, ldq,
                                           ws + code_size, stream));
  if (st != GEMM_OK) return st;
  return run_mx4(dtype, M, N, K, 1.f, ws, ldq, ws + code_size, w_codes, ldw, w_scales, 0.f, Y,
                 ldy, fault, max_pairs, workspaces, stream);
}

gemm_status_t gemm_mx_grad(gemm_mx_format_t fmt, int dtype, gemm_op_t op_a, int dtype_c, int M,
                           int N, int K, float alpha, const void* A, int lda,
                           const void* b_codes, int ldb, const void* b_scales, float beta,
                           void* C, int ldc, cudaStream_t stream) {
  if (!good_format(fmt) || (dtype != 1 && dtype != 2) || !good_op(op_a) ||
      (dtype_c != 0 && dtype_c != dtype) || !good_size(M) || !good_size(N) || !good_size(K))
    return GEMM_ERR_INVALID_ARG;
  if (M == 0 || N == 0) return GEMM_OK;
  const int es = elem_size(dtype_c);
  if (C == nullptr || ldc < N) return GEMM_ERR_INVALID_ARG;
  if (!aligned(C, es)) return GEMM_ERR_MISALIGNED;
  const bool empty = K == 0 || alpha == 0.f;
  // A as stored: `outer` rows of `inner` elements.
  const int inner = op_a == GEMM_OP_T ? M : K, outer = op_a == GEMM_OP_T ? K : M;
  const bool packed = lda == inner && lda % 8 != 0;
  gemm_status_t st;
  if (!empty) {
    if (A == nullptr || lda < (op_a == GEMM_OP_N ? K : M)) return GEMM_ERR_INVALID_ARG;
    if ((st = check_quantized(fmt, N, b_codes, ldb, b_scales)) != GEMM_OK) return st;
    if (packed ? !aligned(A, 2) : (!aligned(A, 16) || lda % 8 != 0)) return GEMM_ERR_MISALIGNED;
    const uint64_t cs = span(M, (long long)N * es, (long long)ldc * es);
    const uint64_t as = op_a == GEMM_OP_N ? span(M, (long long)K * 2, (long long)lda * 2)
                                          : span(K, (long long)M * 2, (long long)lda * 2);
    if (overlap(C, cs, A, as) || overlaps_quantized(C, cs, fmt, K, N, b_codes, ldb, b_scales))
      return GEMM_ERR_INVALID_ARG;
  }
  unsigned* fault;
  int max_pairs;
  if ((st = dgemm::current_device_pairs(&fault, &max_pairs)) != GEMM_OK) return st;
  if (empty) return scale_only(dtype_c, M, N, beta, C, ldc, stream);
  dgemm::StreamWorkspaces workspaces(stream);   // held until everything is queued
  const void* rows = A;
  long long ldr = lda;
  if (packed) {
    ldr = ((long long)lda + 7) / 8 * 8;
    void* p = nullptr;
    if ((st = workspaces.get(dgemm::kWsPack, (size_t)outer * ldr * 2, &p)) != GEMM_OK) return st;
    if ((st = status_of(dgemm::launch_mx_align(A, outer, inner, p, ldr, stream))) != GEMM_OK)
      return st;
    rows = p;
  }
  alignas(64) CUtensorMap tmA, tmB;
  const CUtensorMapDataType dt =
      dtype == 1 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!encode_2d(&tmA, dt, rows, (uint64_t)inner, (uint64_t)outer, (uint64_t)ldr * 2, 64, 64) ||
      !encode_2d(&tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, b_codes, (uint64_t)code_bytes(fmt, N),
                 (uint64_t)K, (uint64_t)ldb, (uint32_t)code_bytes(fmt, 128), dgemm::kMxGradBK,
                 false))
    return GEMM_ERR_LAUNCH;
  dgemm::MxGradParams p;
  p.M = M, p.N = N, p.K = K;
  p.fmt = fmt, p.dtype = dtype, p.op_a = op_a, p.dtype_c = dtype_c;
  p.sb = static_cast<const unsigned char*>(b_scales);
  // (Groups of 8 / 16 tile columns: dX 8192^3 569 / 556 us, 16384 x 4096 x 4096
  // 311 / 304, dW and 4096^3 alike.  The costs are between those of the formats:
  // a k-tile of a whole tile takes 0.57 to 0.61 us with MXFP4, 0.65 to 0.69 with
  // MXINT8 and 0.69 to 0.73 with that in FP16, whatever A's storage and C's type;
  // what counts here are the ratios.)
  p.sched = schedule(M, N, ceil_div(K, dgemm::kMxGradBK), max_pairs, 16, {0.66, 0.50});
  // Terms per sum in tensor memory, which truncates at each step of 16: sums of
  // like terms come out too small, the more the longer they are (FP16, positive
  // terms: 1.4e-6 over 1024, 8.5e-5 over 16384, 3e-3 over 2^19).  FP32 results:
  // 1024 (512 / 256 leave a third / a sixth of the error and take 1.5 to 2.4 % /
  // 7 to 13 % longer).  16-bit ones: 16384, a fifth of FP16's rounding.
  p.seg = (dtype_c == 0 ? 1024 : 16384) / dgemm::kMxGradBK;
  if ((st = partials(p.sched, M, N, workspaces, &p.ws, &p.ldw)) != GEMM_OK) return st;
  p.alpha = alpha, p.beta = beta;
  p.C = C, p.ldc = ldc;
  p.fault = fault, p.timeout_ns = dgemm::wait_bound_ns();
  const int pairs = p.sched.units < max_pairs ? p.sched.units : max_pairs;
  cudaError_t e = dgemm::launch_mx_grad(p, &tmA, &tmB, pairs, stream);
  if (e == cudaSuccess && p.sched.slices > 1)
    e = dgemm::launch_mx_reduce(p.ws, p.sched.slices, M, N, p.ldw, alpha, beta, C, ldc, dtype_c,
                                stream);
  return status_of(e);
}

}  // extern "C"
