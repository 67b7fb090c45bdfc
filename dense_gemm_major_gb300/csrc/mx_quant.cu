// Quantisation to the microscaled formats and back.
//
// Of a block of 32 values x_j: s = floor(log2(max |x_j|)) - emax (clamped),
// codes rn(x_j / 2^s).  Division by a power of two is exact, so the codes do
// not depend on the order of anything.  Both directions are bound by HBM:
// each value is read once and written once.
#include "mx.cuh"

namespace dgemm {
namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void store8(T* dst, const float (&v)[8]) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(dst) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(dst + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(dst) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]),
                                                pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
  }
}

// Row-major X.  A thread takes 8 columns, four threads a block; a warp 256
// columns of one row.  Work item: (row, chunk of 256 columns), chunks
// covering whole tiles of scales so that the padding blocks get theirs.
template <int kFmt, typename T>
__global__ void __launch_bounds__(kThreads)
    mx_quantize_kernel(int R, int K, const T* __restrict__ X, long long ldx, bool vec,
                       unsigned char* __restrict__ codes, long long ldq,
                       unsigned char* __restrict__ scales) {
  wait_prior_grids();
  allow_dependent_grids();
  const int lane = threadIdx.x & 31;
  const int tiles = mx_scale_tiles(K);
  const int chunks = (tiles + 1) / 2;
  const long long items = (long long)R * chunks;
  const long long warps = (long long)gridDim.x * (kThreads / 32);
  for (long long it = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); it < items;
       it += warps) {
    const int r = (int)(it / chunks);
    const int col = (int)(it - (long long)r * chunks) * 256 + lane * 8;
    float v[8];
    const T* src = X + (long long)r * ldx + col;
    if (vec && col + 8 <= K) {
      load8<T>(src, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = col + j < K ? to_f32_any<T>(src[j]) : 0.f;
    }
    unsigned amax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, abs_bits(v[j]));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const unsigned s = mx_scale_byte<kFmt>(amax);
    const float inv = mx_inverse_scale(s);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = s == 255u ? 0.f : v[j] * inv;
    if (col < K) {
      unsigned char* q = codes + (long long)r * ldq;
      if constexpr (kFmt == GEMM_MXFP4)
        *reinterpret_cast<unsigned*>(q + col / 2) = e2m1x8(v);
      else
        *reinterpret_cast<uint2*>(q + col) = int8x8(v);
    }
    const int block = col >> 5;
    if ((lane & 3) == 0 && block < tiles * kMxTileBlocks)
      scales[mx_scale_offset(r, block, tiles)] = (unsigned char)s;
  }
}

// X stored K x R: a thread takes a block of one row (32 values, ldx apart);
// a warp 32 consecutive rows, so that each load is contiguous.
template <int kFmt, typename T>
__global__ void __launch_bounds__(kThreads)
    mx_quantize_t_kernel(int R, int K, const T* __restrict__ X, long long ldx,
                         unsigned char* __restrict__ codes, long long ldq,
                         unsigned char* __restrict__ scales) {
  wait_prior_grids();
  allow_dependent_grids();
  const int lane = threadIdx.x & 31;
  const int tiles = mx_scale_tiles(K);
  const int blocks = tiles * kMxTileBlocks;
  const long long items = (long long)((R + 31) / 32) * blocks;
  const long long warps = (long long)gridDim.x * (kThreads / 32);
  for (long long it = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); it < items;
       it += warps) {
    const int rg = (int)(it / blocks);
    const int block = (int)(it - (long long)rg * blocks);
    const int r = rg * 32 + lane;
    if (r >= R) continue;
    const int k0 = block * kMxBlock;
    float v[32];
    unsigned amax = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      v[j] = k0 + j < K ? to_f32_any<T>(X[(long long)(k0 + j) * ldx + r]) : 0.f;
      amax = max(amax, abs_bits(v[j]));
    }
    const unsigned s = mx_scale_byte<kFmt>(amax);
    const float inv = mx_inverse_scale(s);
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = s == 255u ? 0.f : v[8 * g + j] * inv;
      const int col = k0 + 8 * g;
      if (col < K) {
        unsigned char* q = codes + (long long)r * ldq;
        if constexpr (kFmt == GEMM_MXFP4)
          *reinterpret_cast<unsigned*>(q + col / 2) = e2m1x8(w);
        else
          *reinterpret_cast<uint2*>(q + col) = int8x8(w);
      }
    }
    scales[mx_scale_offset(r, block, tiles)] = (unsigned char)s;
  }
}

// The values of 8 columns per thread.
template <int kFmt, typename T>
__global__ void __launch_bounds__(kThreads)
    mx_dequantize_kernel(int R, int K, const unsigned char* __restrict__ codes, long long ldq,
                         const unsigned char* __restrict__ scales, T* __restrict__ Y,
                         long long ldy, bool vec) {
  wait_prior_grids();
  allow_dependent_grids();
  const int lane = threadIdx.x & 31;
  const int tiles = mx_scale_tiles(K);
  const int chunks = (K + 255) / 256;
  const long long items = (long long)R * chunks;
  const long long warps = (long long)gridDim.x * (kThreads / 32);
  for (long long it = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); it < items;
       it += warps) {
    const int r = (int)(it / chunks);
    const int col = (int)(it - (long long)r * chunks) * 256 + lane * 8;
    if (col >= K) continue;
    const float scale = mx_scale_value(scales[mx_scale_offset(r, col >> 5, tiles)]);
    const unsigned char* q = codes + (long long)r * ldq;
    float v[8];
    if constexpr (kFmt == GEMM_MXFP4) {
      e2m1x8_to_f32(*reinterpret_cast<const unsigned*>(q + col / 2), v);
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(q + col);
      int8x4_to_f32(w.x, v);
      int8x4_to_f32(w.y, v + 4);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= scale;
    T* dst = Y + (long long)r * ldy + col;
    if (vec && col + 8 <= K) {
      store8<T>(dst, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < K) dst[j] = from_f32_any<T>(v[j]);
    }
  }
}

int grid_for(long long items) {
  const long long ctas = (items + kThreads / 32 - 1) / (kThreads / 32);
  return (int)(ctas < 65535 * 8 ? ctas : 65535 * 8);
}

template <typename T>
bool rows16(const T* p, long long ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * (long long)sizeof(T)) % 16 == 0;
}

template <int kFmt, typename T>
cudaError_t quantize_typed(int op, int R, int K, const T* X, long long ldx, unsigned char* codes,
                           long long ldq, unsigned char* scales, cudaStream_t stream) {
  const int tiles = mx_scale_tiles(K);
  if (op == GEMM_OP_N) {
    const long long items = (long long)R * ((tiles + 1) / 2);
    return launch_gemm_kernel(mx_quantize_kernel<kFmt, T>, dim3(grid_for(items)), dim3(kThreads), 0,
                              stream, R, K, X, ldx, rows16(X, ldx), codes, ldq, scales);
  }
  const long long items = (long long)((R + 31) / 32) * tiles * kMxTileBlocks;
  return launch_gemm_kernel(mx_quantize_t_kernel<kFmt, T>, dim3(grid_for(items)), dim3(kThreads),
                            0, stream, R, K, X, ldx, codes, ldq, scales);
}

template <int kFmt, typename T>
cudaError_t dequantize_typed(int R, int K, const unsigned char* codes, long long ldq,
                             const unsigned char* scales, T* Y, long long ldy,
                             cudaStream_t stream) {
  const long long items = (long long)R * ((K + 255) / 256);
  return launch_gemm_kernel(mx_dequantize_kernel<kFmt, T>, dim3(grid_for(items)), dim3(kThreads), 0,
                            stream, R, K, codes, ldq, scales, Y, ldy, rows16(Y, ldy));
}

template <int kFmt>
cudaError_t quantize_fmt(int dtype, int op, int R, int K, const void* X, long long ldx,
                         unsigned char* q, long long ldq, unsigned char* s, cudaStream_t st) {
  if (dtype == 0)
    return quantize_typed<kFmt>(op, R, K, static_cast<const float*>(X), ldx, q, ldq, s, st);
  if (dtype == 1)
    return quantize_typed<kFmt>(op, R, K, static_cast<const __half*>(X), ldx, q, ldq, s, st);
  return quantize_typed<kFmt>(op, R, K, static_cast<const __nv_bfloat16*>(X), ldx, q, ldq, s, st);
}

template <int kFmt>
cudaError_t dequantize_fmt(int dtype, int R, int K, const unsigned char* q, long long ldq,
                           const unsigned char* s, void* Y, long long ldy, cudaStream_t st) {
  if (dtype == 0)
    return dequantize_typed<kFmt>(R, K, q, ldq, s, static_cast<float*>(Y), ldy, st);
  if (dtype == 1)
    return dequantize_typed<kFmt>(R, K, q, ldq, s, static_cast<__half*>(Y), ldy, st);
  return dequantize_typed<kFmt>(R, K, q, ldq, s, static_cast<__nv_bfloat16*>(Y), ldy, st);
}

}  // namespace

cudaError_t launch_mx_quantize(int fmt, int dtype, int op, int R, int K, const void* X,
                               long long ldx, void* codes, long long ldq, void* scales,
                               cudaStream_t stream) {
  unsigned char* q = static_cast<unsigned char*>(codes);
  unsigned char* s = static_cast<unsigned char*>(scales);
  return fmt == GEMM_MXFP4 ? quantize_fmt<GEMM_MXFP4>(dtype, op, R, K, X, ldx, q, ldq, s, stream)
                           : quantize_fmt<GEMM_MXINT8>(dtype, op, R, K, X, ldx, q, ldq, s, stream);
}

cudaError_t launch_mx_dequantize(int fmt, int dtype, int R, int K, const void* codes,
                                 long long ldq, const void* scales, void* Y, long long ldy,
                                 cudaStream_t stream) {
  const unsigned char* q = static_cast<const unsigned char*>(codes);
  const unsigned char* s = static_cast<const unsigned char*>(scales);
  return fmt == GEMM_MXFP4 ? dequantize_fmt<GEMM_MXFP4>(dtype, R, K, q, ldq, s, Y, ldy, stream)
                           : dequantize_fmt<GEMM_MXINT8>(dtype, R, K, q, ldq, s, Y, ldy, stream);
}

}  // namespace dgemm
