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

// The value in a word as loaded: half i of a pair of 16-bit ones, or FP32.
template <typename T>
__device__ __forceinline__ float value_of(unsigned w, int i) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(w);
  } else {
    const float2 f = pair_to_f32<T>(w);
    return i == 0 ? f.x : f.y;
  }
}
// Two values as a pair of a 16-bit type (never called for FP32).
template <typename T>
__device__ __forceinline__ unsigned pack2_any(float lo, float hi) {
  if constexpr (sizeof(T) == 2) return pack2<T>(lo, hi);
  return 0u;
}

// Row-major X.  A thread takes 8 columns, four threads a block, a warp 256
// columns of a row at a time and kStep such pieces in a row, their loads in
// flight together: HBM's latency needs some 40 KB of them per SM.  A CTA has
// kThreads / 32 rows; pieces cover whole tiles of scales, so that the padding
// blocks get theirs.
constexpr int kStep = 4;
constexpr int kRowsPerCta = kThreads / 32;

template <int kFmt, typename T>
__global__ void __launch_bounds__(kThreads)
    mx_quantize_kernel(int R, int K, const T* __restrict__ X, long long ldx, bool vec,
                       unsigned char* __restrict__ codes, long long ldq,
                       unsigned char* __restrict__ scales) {
  wait_prior_grids();
  allow_dependent_grids();
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * kRowsPerCta + (threadIdx.x >> 5);
  if (r >= R) return;
  const int tiles = mx_scale_tiles(K);
  const int pieces = (tiles + 1) / 2;
  const T* row = X + (long long)r * ldx;
  unsigned char* q = codes + (long long)r * ldq;
  unsigned char* srow = scales + mx_scale_offset(r, (lane >> 2) & 3, tiles);
  for (int p0 = blockIdx.y * kStep; p0 < pieces; p0 += gridDim.y * kStep) {
    float v[kStep][8];
    // (The two ways apart, so that the compiler keeps all loads of the first
    // in flight.)
    if (vec && (p0 + kStep) * 256 <= K) {
#pragma unroll
      for (int i = 0; i < kStep; ++i) load8<T>(row + (p0 + i) * 256 + lane * 8, v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        const int col = (p0 + i) * 256 + lane * 8;
        if (vec && col + 8 <= K) {
          load8<T>(row + col, v[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = col + j < K ? to_f32_any<T>(row[col + j]) : 0.f;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      if (p0 + i >= pieces) break;
      const int col = (p0 + i) * 256 + lane * 8;
      unsigned amax = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = max(amax, abs_bits(v[i][j]));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const unsigned s = mx_scale_byte<kFmt>(amax);
      const float inv = mx_inverse_scale(s);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= inv;
      if (col < K) {
        if constexpr (kFmt == GEMM_MXFP4) {
          *reinterpret_cast<unsigned*>(q + col / 2) = s == 255u ? 0u : e2m1x8(v[i]);
        } else {
          const uint2 c = int8x8(v[i], int8_clamps(amax, inv));
          *reinterpret_cast<uint2*>(q + col) = s == 255u ? make_uint2(0u, 0u) : c;
        }
      }
      const int tile = (p0 + i) * 2 + (lane >> 4);
      if ((lane & 3) == 0 && tile < tiles)
        srow[(long long)tile * kMxTileBytes] = (unsigned char)s;
    }
  }
}

// X stored K x R.  A CTA takes 32 V rows and 256 columns (V = 2 for 16-bit
// types, whose two rows travel in one load), a warp one block of them: its
// loads are contiguous along R.  The codes of the CTA meet in shared memory,
// so that they leave as 128 (MXFP4) or 256 contiguous bytes of a row, and the
// scales as words of four.
template <int kFmt, typename T>
struct TLayout {
  static constexpr int V = sizeof(T) == 4 ? 1 : 2;
  static constexpr int kRows = 32 * V;
  static constexpr int kBlockBytes = kFmt == GEMM_MXFP4 ? 16 : 32;   // codes of a block
  static constexpr int kRowBytes = 8 * kBlockBytes;
  static constexpr int kPitch = kRowBytes + 16;                      // (bank conflicts)
};

template <int kFmt, typename T>
__global__ void __launch_bounds__(kThreads)
    mx_quantize_t_kernel(int R, int K, const T* __restrict__ X, long long ldx, bool vec,
                         unsigned char* __restrict__ codes, long long ldq,
                         unsigned char* __restrict__ scales) {
  using L = TLayout<kFmt, T>;
  __shared__ __align__(16) unsigned char scode[L::kRows * L::kPitch];
  __shared__ __align__(4) unsigned char sscale[L::kRows * 8];
  wait_prior_grids();
  allow_dependent_grids();
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int tiles = mx_scale_tiles(K);
  const int r0 = blockIdx.x * L::kRows;
  const int pieces = (tiles + 1) / 2;
  for (int piece = blockIdx.y; piece < pieces; piece += gridDim.y) {
    const int k0 = piece * 256 + warp * kMxBlock;
    const int r = r0 + lane * L::V;
    // The block's values as loaded (pairs of 16-bit ones stay packed: half the
    // registers, twice the CTAs per SM).
    unsigned raw[32];
    if ((L::V == 1 || vec) && r + L::V <= R && k0 + kMxBlock <= K) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        raw[j] = *reinterpret_cast<const unsigned*>(X + (long long)(k0 + j) * ldx + r);
    } else if constexpr (L::V == 1) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        raw[j] = k0 + j < K && r < R
                     ? *reinterpret_cast<const unsigned*>(X + (long long)(k0 + j) * ldx + r)
                     : 0u;
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        unsigned h[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          h[i] = k0 + j < K && r + i < R
                     ? reinterpret_cast<const unsigned short*>(X)[(long long)(k0 + j) * ldx + r + i]
                     : 0u;
        raw[j] = h[0] | (h[1] << 16);
      }
    }
#pragma unroll
    for (int i = 0; i < L::V; ++i) {
      unsigned amax = 0;
#pragma unroll
      for (int j = 0; j < 32; ++j) amax = max(amax, abs_bits(value_of<T>(raw[j], i)));
      const unsigned s = mx_scale_byte<kFmt>(amax);
      const float inv = mx_inverse_scale(s);
      const bool clamp = kFmt == GEMM_MXINT8 && int8_clamps(amax, inv);
      const int row = lane * L::V + i;
      uint4* dst = reinterpret_cast<uint4*>(scode + row * L::kPitch + warp * L::kBlockBytes);
      unsigned w[8];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = value_of<T>(raw[8 * g + j], i) * inv;
        if constexpr (kFmt == GEMM_MXFP4) {
          w[g] = s == 255u ? 0u : e2m1x8(x);
        } else {
          const uint2 c = int8x8(x, clamp);
          w[2 * g] = s == 255u ? 0u : c.x;
          w[2 * g + 1] = s == 255u ? 0u : c.y;
        }
      }
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      if constexpr (kFmt == GEMM_MXINT8) dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      sscale[row * 8 + warp] = (unsigned char)s;
    }
    __syncthreads();
    // In 16-byte chunks; a ragged piece ends with words, after its last group of
    // 8 columns.  (The two ways apart: together they took 8 % longer.)
    unsigned char* const q = codes + (long long)r0 * ldq + (long long)piece * L::kRowBytes;
    constexpr int kChunks = L::kRowBytes / 16;
    if (K - piece * 256 > 248) {
#pragma unroll
      for (int i = threadIdx.x; i < L::kRows * kChunks; i += kThreads) {
        const int row = i / kChunks, at = i % kChunks * 16;
        if (r0 + row < R)
          *reinterpret_cast<uint4*>(q + row * ldq + at) =
              *reinterpret_cast<const uint4*>(scode + row * L::kPitch + at);
      }
    } else {
      const int left = (K - piece * 256 + 7) / 8 * (L::kBlockBytes / 4);
#pragma unroll 1
      for (int i = threadIdx.x; i < L::kRows * kChunks; i += kThreads) {
        const int row = i / kChunks, at = i % kChunks * 16;
        if (r0 + row >= R) continue;
        unsigned char* dst = q + row * ldq + at;
        const unsigned char* src = scode + row * L::kPitch + at;
        if (at + 16 <= left) {
          *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
        } else {
#pragma unroll 1
          for (int j = 0; at + j < left; j += 4)
            *reinterpret_cast<unsigned*>(dst + j) = *reinterpret_cast<const unsigned*>(src + j);
        }
      }
    }
    for (int i = threadIdx.x; i < L::kRows * 2; i += kThreads) {
      const int row = i >> 1, tile = piece * 2 + (i & 1);
      if (r0 + row < R && tile < tiles)
        *reinterpret_cast<unsigned*>(scales + mx_scale_offset(r0 + row, tile * 4, tiles)) =
            *reinterpret_cast<const unsigned*>(sscale + row * 8 + (i & 1) * 4);
    }
    __syncthreads();
  }
}

// 2, 4 or 8 bytes of codes, aligned to as many, as one or two words.
template <int kBytes>
__device__ __forceinline__ void load_codes(const unsigned char* c, unsigned* w) {
  if constexpr (kBytes == 2) {
    w[0] = *reinterpret_cast<const unsigned short*>(c);
  } else if constexpr (kBytes == 4) {
    w[0] = *reinterpret_cast<const unsigned*>(c);
  } else {
    const uint2 x = *reinterpret_cast<const uint2*>(c);
    w[0] = x.x;
    w[1] = x.y;
  }
}

// As mx_quantize_kernel, the other way.  A thread's 8 columns of a piece are
// consecutive for 16-bit results and two groups of four, 128 apart, for FP32,
// so that a warp's 16-byte stores are contiguous.
template <int kFmt, typename T>
__global__ void __launch_bounds__(kThreads)
    mx_dequantize_kernel(int R, int K, const unsigned char* __restrict__ codes, long long ldq,
                         const unsigned char* __restrict__ scales, T* __restrict__ Y,
                         long long ldy, bool vec) {
  constexpr int G = sizeof(T) == 4 ? 2 : 1, W = 8 / G;    // groups of W columns,
  constexpr int kBytes = kFmt == GEMM_MXFP4 ? W / 2 : W;   // of this many bytes
  wait_prior_grids();
  allow_dependent_grids();
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * kRowsPerCta + (threadIdx.x >> 5);
  if (r >= R) return;
  const int tiles = mx_scale_tiles(K);
  const int pieces = (K + 255) / 256;
  const unsigned char* q = codes + (long long)r * ldq;
  const unsigned char* srow = scales + mx_scale_offset(r, 0, tiles);
  T* row = Y + (long long)r * ldy;
  for (int p0 = blockIdx.y * kStep; p0 < pieces; p0 += gridDim.y * kStep) {
    unsigned w[kStep][2];
    unsigned s[kStep][G];
    // (The two ways apart, as above.)
    if ((p0 + kStep) * 256 <= K) {
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        w[i][1] = 0u;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int col = (p0 + i) * 256 + g * 128 + lane * W;
          load_codes<kBytes>(q + (kFmt == GEMM_MXFP4 ? col / 2 : col), &w[i][g]);
          s[i][g] = srow[(long long)(col >> 7) * kMxTileBytes + ((col >> 5) & 3)];
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kStep; ++i) {
        w[i][0] = w[i][1] = 0u;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const int col = (p0 + i) * 256 + g * 128 + lane * W;
          const unsigned char* c = q + (kFmt == GEMM_MXFP4 ? col / 2 : col);
          s[i][g] = 0u;
          if (col >= K) continue;
          s[i][g] = srow[(long long)(col >> 7) * kMxTileBytes + ((col >> 5) & 3)];
          if (col + W <= K) {
            load_codes<kBytes>(c, &w[i][g]);
          } else {   // nothing past a row's last code is read
            const int bytes = kFmt == GEMM_MXFP4 ? (K - col + 1) / 2 : K - col;
#pragma unroll
            for (int j = 0; j < kBytes; ++j)
              if (j < bytes) w[i][g + j / 4] |= (unsigned)c[j] << (8 * (j % 4));
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      float v[8];
      if constexpr (kFmt == GEMM_MXFP4) {
        e2m1x8_to_f32(G == 1 ? w[i][0] : w[i][0] | (w[i][1] << 16), v);
      } else {
        int8x4_to_f32(w[i][0], v);
        int8x4_to_f32(w[i][1], v + 4);
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int col = (p0 + i) * 256 + g * 128 + lane * W;
        const float scale = mx_scale_value(s[i][g]);
#pragma unroll
        for (int j = 0; j < W; ++j) v[g * W + j] *= scale;
        if (vec && col + W <= K) {
          if constexpr (G == 1)
            *reinterpret_cast<uint4*>(row + col) =
                make_uint4(pack2_any<T>(v[0], v[1]), pack2_any<T>(v[2], v[3]),
                           pack2_any<T>(v[4], v[5]), pack2_any<T>(v[6], v[7]));
          else
            *reinterpret_cast<float4*>(row + col) =
                make_float4(v[g * W], v[g * W + 1], v[g * W + 2], v[g * W + 3]);
        } else {
#pragma unroll
          for (int j = 0; j < W; ++j)
            if (col + j < K) row[col + j] = from_f32_any<T>(v[g * W + j]);
        }
      }
    }
  }
}

// CTAs of `rows` rows each, and along K of `step` pieces of 256 columns.
dim3 grid_for(int R, int rows, int pieces, int step) {
  const int y = (pieces + step - 1) / step;
  return dim3((unsigned)((R + (long long)rows - 1) / rows), (unsigned)(y < 65535 ? y : 65535));
}

template <typename T>
bool rows16(const T* p, long long ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * (long long)sizeof(T)) % 16 == 0;
}

template <int kFmt, typename T>
cudaError_t quantize_typed(int op, int R, int K, const T* X, long long ldx, unsigned char* codes,
                           long long ldq, unsigned char* scales, cudaStream_t stream) {
  const int pieces = (mx_scale_tiles(K) + 1) / 2;
  if (op == GEMM_OP_N)
    return launch_gemm_kernel(mx_quantize_kernel<kFmt, T>, grid_for(R, kRowsPerCta, pieces, kStep),
                              dim3(kThreads), 0, stream, R, K, X, ldx, rows16(X, ldx), codes, ldq,
                              scales);
  const bool vec = (reinterpret_cast<uintptr_t>(X) & 3u) == 0 && ldx % 2 == 0;
  return launch_gemm_kernel(mx_quantize_t_kernel<kFmt, T>,
                            grid_for(R, TLayout<kFmt, T>::kRows, pieces, 1), dim3(kThreads), 0,
                            stream, R, K, X, ldx, vec, codes, ldq, scales);
}

template <int kFmt, typename T>
cudaError_t dequantize_typed(int R, int K, const unsigned char* codes, long long ldq,
                             const unsigned char* scales, T* Y, long long ldy,
                             cudaStream_t stream) {
  return launch_gemm_kernel(mx_dequantize_kernel<kFmt, T>,
                            grid_for(R, kRowsPerCta, (K + 255) / 256, kStep), dim3(kThreads), 0,
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
