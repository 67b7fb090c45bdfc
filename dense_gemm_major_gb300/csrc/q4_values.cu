// 4-bit weights with group scales in 16 bits, for products of many rows: what a value
// takes is to be read and written once, 2.5 bytes and its share of the scales.
#include "q4.cuh"

namespace dgemm {
namespace {

// Each thread: the 32 codes of 16 bytes, which share a scale.  A block takes 32 rows x
// 8 such chunks, a warp's lanes 8 rows x 4 chunks.
template <typename T>
__global__ void __launch_bounds__(256)
    q4_values_kernel(int group, long long tiles_n, int N, int K, int scale_n,
                     const unsigned char* codes, int ldq, long long stride_q, const T* scales,
                     const unsigned char* zeros, const int* offsets, T* D, long long ldd) {
  wait_prior_grids();
  allow_dependent_grids();
  const int chunks = (K + 31) / 32, groups = q4_groups(K, group);
  const int e = (int)(blockIdx.x / tiles_n);
  if (offsets != nullptr && offsets[e + 1] <= offsets[e]) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = (int)(blockIdx.x - e * tiles_n) * 32 + (warp & 3) * 8 + (lane >> 2);
  if (n >= N) return;
  const unsigned char* const q_row = codes + e * stride_q + (long long)n * ldq;
  const long long s_row = (long long)e * groups * scale_n + n;
  T* const d_row = D + ((long long)e * N + n) * ldd;
  for (int c = (int)blockIdx.y * 8 + (warp >> 2) * 4 + (lane & 3); c < chunks;
       c += (int)gridDim.y * 8) {
    uint4 w = make_uint4(0, 0, 0, 0);
    if (c * 32ll + 32 <= K) {
      w = *reinterpret_cast<const uint4*>(q_row + (long long)c * 16);
    } else {   // nothing past the row's last code is read
      unsigned char* const bytes = reinterpret_cast<unsigned char*>(&w);
      for (int b = 0; 2 * b < K - c * 32; ++b) bytes[b] = q_row[(long long)c * 16 + b];
    }
    const long long at = s_row + (long long)(c * 32ll / group) * scale_n;
    const float s = elem_to_f32<T>(scales[at]);
    const float z = zeros != nullptr ? (float)(zeros[at] & 15) : 8.f;
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
    T* const to = d_row + (long long)c * 32;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (c * 32ll + j * 8 >= K) break;     // (ldd has room for whole groups of 8)
      uint32_t v[4];
#pragma unroll
      for (int h = 0; h < 4; ++h)
        v[h] = pack2<T>(((float)((q[j] >> (8 * h)) & 15u) - z) * s,
                        ((float)((q[j] >> (8 * h + 4)) & 15u) - z) * s);
      *reinterpret_cast<uint4*>(to + j * 8) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
}

}  // namespace

cudaError_t launch_q4_values(int dtype, int group, int experts, int N, int K, int scale_n,
                             const unsigned char* codes, int ldq, long long stride_q,
                             const void* scales, const unsigned char* zeros, const int* offsets,
                             void* D, long long ldd, cudaStream_t stream) {
  const long long tiles_n = (N + 31ll) / 32;
  const int parts = (K + 255) / 256;
  const dim3 grid((unsigned)(experts * tiles_n), (unsigned)(parts < 65535 ? parts : 65535));
  if (dtype == 1)
    return launch_gemm_kernel(q4_values_kernel<__half>, grid, dim3(256), 0, stream, group, tiles_n,
                              N, K, scale_n, codes, ldq, stride_q,
                              static_cast<const __half*>(scales), zeros, offsets,
                              static_cast<__half*>(D), ldd);
  return launch_gemm_kernel(q4_values_kernel<__nv_bfloat16>, grid, dim3(256), 0, stream, group,
                            tiles_n, N, K, scale_n, codes, ldq, stride_q,
                            static_cast<const __nv_bfloat16*>(scales), zeros, offsets,
                            static_cast<__nv_bfloat16*>(D), ldd);
}

}  // namespace dgemm
