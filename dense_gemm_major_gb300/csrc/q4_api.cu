// C-ABI entry point of the products with 4-bit weights and group scales: argument
// checks, choice between the kernel for few rows and a product with the weights in
// 16 bits, launch.  See include/dense_gemm_q4.h.
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "group.h"
#include "group_operands.h"
#include "q4.h"
#include "workspace.h"

namespace {

using namespace dgemm::api;

inline bool good_size(int n) { return n >= 0 && n <= GEMM_GROUP_MAX_SIZE; }

struct Q4Call {
  int dtype, group, rows, N, K, experts;
  Operand x;
  const unsigned char* codes;
  int ldq;
  const void* scales;
  const unsigned char* zeros;
  const int* offsets;
  void* Y;
  int ldy;
  unsigned* fault;
  int pairs;
  int matrices() const { return experts == 0 ? 1 : experts; }
};

// Which kernel, by the rows (of an expert) to expect.
//
// Few: mma.sync on registers.  Against the tcgen05 kernel, us, BF16 and groups of 128 / FP16
// and groups of 64 / BF16 and 32: 8 rows 1024 x 1024 2.7 / 2.7 / 2.9 and 3.9 / 4.2 / 4.2, 4096 x
// 4096 5.6 / 5.7 / 6.5 and 6.9 / 7.3 / 7.4, 8192 x 8192 11.9 / 12.6 / 14.8 and 13.6 / 14.9 / 15.3,
// 14336 x 4096 10.8 / 11.6 / 13.8 and 13.8 / 16.2 / 16.1; 16 rows 1024 x 1024 3.4 / 3.6 / 3.8 and
// 4.0 / 4.2 / 4.4, 2048 x 8192 6.7 and 8.5, 4096 x 4096 6.9 / 7.4 / 8.2 and 7.1 / 7.4 / 7.5; but
// 8192 x 8192 14.9 / 16.8 / 19.2 and 13.6 / 14.9 / 15.4.  Of experts (2048 x 2048, groups of
// 128): 8 rows each of 8 8.6 / 10.3, of 32 23.6 / 26.1, of 64 39.6 / 42.7, 5 of 8 8.5 / 10.2;
// but 16 each of 32 36.2 / 26.8.
constexpr int kFewRows = 8, kFewRowsSmall = 16;
constexpr long long kFewSmall = 1ll << 24;         // weights
bool few_rows(const Q4Call& c, int expect) {
  return expect <= (c.experts == 0 && (long long)c.N * c.K <= kFewSmall ? kFewRowsSmall
                                                                        : kFewRows);
}
// Rows: tcgen05, each 128 rows' units converting the weights for themselves.  Against the
// product with the weights in 16 bits, us, one after the other under the power limit, groups
// of 128: 1024 rows 4096 x 4096 29.7 / 37.1, 2048 55.7 / 57.6 (of 32: 61.3 / 57.9) and 8192 x
// 8192 189 / 220, 8 experts of 1024 rows each, 2048 x 2048, 61 / 75, of 2048, 4096 x 4096, 399 /
// 418; but 4096 rows 4096 x 4096 102.2 / 100.7, 8192 x 8192 372 / 381; singly 8192 rows 4096 x
// 4096 176 / 162, 8 experts of 4096, 2048 x 2048, 207 / 181.
constexpr int kCodeRows = 2048;

// The product by one of the kernels that read the codes.  (Not done: terms beyond what a
// sum in tensor memory, which truncates at each step, should have; see segment().  BF16
// rounds eight times as coarsely.)
bool run_codes(const Q4Call& c, int expect, cudaStream_t stream, gemm_status_t* st) {
  const bool few = few_rows(c, expect);
  dgemm::Q4FewParams p;
  p.rows = c.rows, p.N = c.N, p.K = c.K, p.group = c.group;
  p.experts = c.experts, p.offsets = c.offsets;
  if (few)
    p.tile_rows = expect <= 8 ? 8 : 16;
  else   // (An expert with more rows than a tile has its weights converted again.)
    p.tile_rows = dgemm::q4_rows_tile(c.experts == 0 ? expect : 2 * expect);
  p.slots = c.experts == 0 ? ceil_div(c.rows, p.tile_rows)
                           : c.rows / p.tile_rows + (c.experts < c.rows ? c.experts : c.rows);
  // CTAs that share a tile's K: as many (a cluster of at most 8) as keep one wave, each with a
  // slot of codes at least, and no more than shorten the longest share.  (Of 16 clusters of 8
  // on 152 SMs one has to wait: 33 x 2048 x 4096 11.4 us, in clusters of 4 6.9.  Not only powers
  // of two: 2 x 5120 x 13824 16.8 -> 12.7 us, 40 rows 19.7 -> 15.6, 2 x 2560 x 2560 4.2 -> 3.7.)
  const int tile_n = few ? dgemm::kQ4TileN : dgemm::kQ4RowsTileN;
  const long long tiles = (long long)ceil_div(c.N, tile_n) * p.slots;
  const int nk = ceil_div(c.K, few ? dgemm::kQ4BK : 2 * dgemm::kQ4RowsBK);
  const int room = 2 * c.pairs * (few ? 2 : 1);
  p.max_ctas = room;
  for (p.split = nk < 8 ? nk : 8; p.split > 1; --p.split) {
    if (p.split * tiles > room || ceil_div(nk, p.split) == ceil_div(nk, p.split - 1)) continue;
    if (tiles <= (few ? dgemm::q4_few_clusters(p.split) : dgemm::q4_rows_clusters(p.split))) break;
  }
  const long long terms = ceil_div(nk, p.split) * 2ll * dgemm::kQ4RowsBK;
  if (!few && terms > (long long)segment(c.dtype) * dgemm::kGroupBK * (c.dtype == 2 ? 8 : 1))
    return false;
  p.scales = c.scales, p.zeros = c.zeros;
  p.Y = c.Y, p.ldy = c.ldy;
  p.fault = c.fault, p.timeout_ns = dgemm::wait_bound_ns();
  alignas(64) CUtensorMap tmQ, tmX;
  const cuuint64_t dims[3] = {(cuuint64_t)((c.K + 1ll) / 2), (cuuint64_t)c.N,
                              (cuuint64_t)c.matrices()};
  const cuuint64_t strides[2] = {(cuuint64_t)c.ldq, (cuuint64_t)c.N * c.ldq};
  const cuuint32_t box[3] = {128, (cuuint32_t)tile_n, 1};
  if (!encode_tiled(&tmQ, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, c.codes, dims, strides, box) ||
      !encode_rows(&tmX, c.dtype, c.x, (uint32_t)p.tile_rows))
    *st = GEMM_ERR_LAUNCH;
  else
    *st = status_of(few ? dgemm::launch_q4_few(c.dtype, p, &tmQ, &tmX, stream)
                        : dgemm::launch_q4_rows(c.dtype, p, &tmQ, &tmX, stream));
  return true;
}

// The product with the weights in 16 bits, in parts of them that fit the workspace:
// some experts, or some columns of Y.
gemm_status_t run_values(const Q4Call& c, dgemm::StreamWorkspaces& workspaces,
                         cudaStream_t stream) {
  const long long ldd = ((long long)c.K + 7) / 8 * 8, groups = dgemm::q4_groups(c.K, c.group);
  long long fit = GEMM_Q4_WORKSPACE / (ldd * 2);       // rows of W
  if (fit < 1) fit = 1;
  const bool whole = fit >= c.N;                        // matrices at a time, or parts of one
  const int part = whole ? c.N : (int)(fit >= 256 ? fit / 256 * 256 : fit);
  int together = whole ? (int)(fit / c.N < c.matrices() ? fit / c.N : c.matrices()) : 1;
  void* d = nullptr;
  gemm_status_t st =
      workspaces.get(dgemm::kWsValues, (size_t)together * part * ldd * 2, &d);
  if (st != GEMM_OK) return st;
  dgemm::GroupParams p;
  p.kind = dgemm::kGroupForward;
  p.tile_rows = dgemm::kGroupTile;
  p.rows = c.rows, p.M = 0, p.K = c.K, p.per_group = 0;
  p.zmul = 1;
  p.seg = segment(c.dtype);
  p.alpha = 1.f, p.beta = 0.f;
  p.ldc = c.ldy, p.stride_c = 0;
  p.fault = c.fault, p.timeout_ns = dgemm::wait_bound_ns();
  alignas(64) CUtensorMap tmM, tmN, tmN16;
  if (!encode_rows(&tmN, c.dtype, c.x, 128) || !encode_rows(&tmN16, c.dtype, c.x, 16))
    return GEMM_ERR_LAUNCH;
  for (int e = 0; e < c.matrices(); e += together) {
    const int n = c.matrices() - e < together ? c.matrices() - e : together;
    for (int n0 = 0; n0 < c.N; n0 += part) {
      const int cols = c.N - n0 < part ? c.N - n0 : part;
      const long long first = (long long)e * groups * c.N + n0;   // scale
      st = status_of(dgemm::launch_q4_values(
          c.dtype, c.group, n, cols, c.K, c.N, c.codes + ((long long)e * c.N + n0) * c.ldq, c.ldq,
          (long long)c.N * c.ldq, static_cast<const char*>(c.scales) + first * 2,
          c.zeros == nullptr ? nullptr : c.zeros + first,
          c.offsets == nullptr ? nullptr : c.offsets + e, d, ldd, stream));
      if (st != GEMM_OK) return st;
      const Operand w{d, c.K, cols, ldd, n, (long long)cols * ldd, false};
      if (!encode_matrices(&tmM, c.dtype, w)) return GEMM_ERR_LAUNCH;
      p.groups = n, p.first_group = e, p.N = cols, p.offsets = c.offsets;
      p.C = static_cast<char*>(c.Y) + (long long)n0 * 2;
      const long long most = dgemm::group_units(c.rows, n, cols, p.tile_rows);
      st = status_of(dgemm::launch_group(c.dtype, c.dtype, p, &tmM, &tmN, &tmN16,
                                         (int)(most < c.pairs ? most : c.pairs), stream));
      if (st != GEMM_OK) return st;
    }
  }
  return GEMM_OK;
}

}  // namespace

extern "C" gemm_status_t gemm_q4_linear(int dtype, int group, int rows, int N, int K, int experts,
                                        const void* X, int ldx, const void* codes, int ldq,
                                        const void* scales, const void* zeros,
                                        const int* offsets, void* Y, int ldy,
                                        cudaStream_t stream) {
  if ((dtype != 1 && dtype != 2) || group < 32 || group % 32 != 0 || !good_size(rows) ||
      !good_size(N) || !good_size(K) || experts < 0 || experts > GEMM_GROUP_MAX_GROUPS ||
      (experts == 0) != (offsets == nullptr))
    return GEMM_ERR_INVALID_ARG;
  if (rows == 0 || N == 0) return GEMM_OK;
  if (Y == nullptr || ldy < N) return GEMM_ERR_INVALID_ARG;
  if (!aligned(Y, 2) || !aligned(offsets, 4)) return GEMM_ERR_MISALIGNED;
  Q4Call c{dtype, group, rows, N, K, experts, Operand{X, K, rows, ldx, 1, 0, false},
           static_cast<const unsigned char*>(codes), ldq, scales,
           static_cast<const unsigned char*>(zeros), offsets, Y, ldy, nullptr, 0};
  const uint64_t ys = span(rows, (long long)N * 2, (long long)ldy * 2);
  gemm_status_t st;
  if (overlap(Y, ys, offsets, offsets == nullptr ? 0 : (uint64_t)(experts + 1) * 4))
    return GEMM_ERR_INVALID_ARG;
  if (K > 0) {
    if (codes == nullptr || scales == nullptr || ldq < (K + 1ll) / 2) return GEMM_ERR_INVALID_ARG;
    if (!aligned(codes, 16) || ldq % 16 != 0 || !aligned(scales, 2)) return GEMM_ERR_MISALIGNED;
    if ((st = c.x.check()) != GEMM_OK) return st;
    const long long all = (long long)c.matrices() * N, g = dgemm::q4_groups(K, group);
    if (overlap(Y, ys, X, c.x.bytes()) ||
        overlap(Y, ys, codes, span(all, (K + 1ll) / 2, ldq)) ||
        overlap(Y, ys, scales, (uint64_t)(all * g * 2)) ||
        overlap(Y, ys, zeros, (uint64_t)(all * g)))
      return GEMM_ERR_INVALID_ARG;
  } else {
    // No terms: the groups' rows become zeros.
    if (experts != 0)
      return gemm_grouped(dtype, GEMM_OP_T, dtype, rows, N, 0, experts, 1.f, nullptr, 0, nullptr,
                          0, 0, offsets, 0.f, Y, ldy, stream);
  }
  if ((st = dgemm::current_device_pairs(&c.fault, &c.pairs)) != GEMM_OK) return st;
  if (K == 0) return status_of(dgemm::launch_scale_c(Y, rows, N, ldy, dtype, 0.f, stream));
  dgemm::StreamWorkspaces workspaces(stream);   // held until everything is queued
  Operand none{nullptr, 0, 0, 0, 1, 0, false};
  if ((st = align_operands(c.x, none, workspaces, stream)) != GEMM_OK) return st;
  const int expect = experts == 0 ? rows : ceil_div(rows, experts);
  if (expect <= kCodeRows && run_codes(c, expect, stream, &st)) return st;
  return run_values(c, workspaces, stream);
}
