// Before and after the products: the copy of a packed 16-bit operand to rows
// that TMA can address, and the sum of the FP32 partial results of a product
// split along K, with its epilogue: C := alpha * sum + beta * C, slices added
// in order.  The partial results have just been written and are read from L2.
#include "mx.cuh"

namespace dgemm {
namespace {

constexpr int kThreads = 256;

// A thread takes four columns of a row, all slices' loads in flight together
// in groups of kStep.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    mx_reduce_kernel(const float* __restrict__ ws, int slices, int M, int N, long long ldw,
                     float alpha, float beta, T* __restrict__ C, long long ldc, bool vec) {
  constexpr int kStep = 4;
  wait_prior_grids();
  allow_dependent_grids();
  const int groups = (N + 127) / 128;
  const int rg = blockIdx.x / groups;
  const int row = rg * (kThreads / 32) + (threadIdx.x >> 5);
  const int col = ((blockIdx.x - rg * groups) * 32 + (threadIdx.x & 31)) * 4;
  if (row >= M || col >= N) return;
  const float* src = ws + (long long)row * ldw + col;
  const long long stride = (long long)M * ldw;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < slices; s0 += kStep) {
    float4 v[kStep];
#pragma unroll
    for (int i = 0; i < kStep; ++i)
      v[i] = s0 + i < slices ? *reinterpret_cast<const float4*>(src + (s0 + i) * stride)
                             : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      sum.x += v[i].x;
      sum.y += v[i].y;
      sum.z += v[i].z;
      sum.w += v[i].w;
    }
  }
  T* c = C + (long long)row * ldc + col;
  float x[4] = {alpha * sum.x, alpha * sum.y, alpha * sum.z, alpha * sum.w};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (beta != 0.f && col + j < N) x[j] = fmaf(beta, to_f32_any<T>(c[j]), x[j]);
  if (vec && col + 4 <= N) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4*>(c) = make_float4(x[0], x[1], x[2], x[3]);
    else
      *reinterpret_cast<uint2*>(c) = make_uint2(pack2<T>(x[0], x[1]), pack2<T>(x[2], x[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (col + j < N) c[j] = from_f32_any<T>(x[j]);
  }
}

// D (rows of ldd elements, 16-byte aligned) := S, rows x cols packed 16-bit
// elements at any even address.  A thread takes 8 columns of a row of D: one
// 16-byte store, and four words of S, or three and the two elements around
// them where S is odd there.  Bound by HBM and L2: S is read and D written
// once (8192 x 4097, 67 MB each way: 22 us, 6.1 TB/s).
__global__ void __launch_bounds__(kThreads)
    mx_align_kernel(const unsigned short* __restrict__ S, long long rows, int cols,
                    unsigned short* __restrict__ D, long long ldd) {
  wait_prior_grids();
  allow_dependent_grids();
  const unsigned groups = (unsigned)(ldd / 8);
  const long long total = rows * groups;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (long long)gridDim.x * kThreads) {
    const long long r = i / groups;
    const int c = (int)(i - r * groups) * 8;
    const unsigned short* src = S + r * cols + c;
    uint4 v;
    if (c + 8 <= cols) {
      const unsigned* w;
      if ((reinterpret_cast<uintptr_t>(src) & 2u) == 0) {
        w = reinterpret_cast<const unsigned*>(src);
        v = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        w = reinterpret_cast<const unsigned*>(src + 1);
        const unsigned a = src[0], b = w[0], d = w[1], e = w[2], f = src[7];
        v = make_uint4(a | (b << 16), __funnelshift_r(b, d, 16), __funnelshift_r(d, e, 16),
                       (e >> 16) | (f << 16));
      }
    } else {
      unsigned h[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = c + j < cols ? src[j] : 0u;
      v = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16),
                     h[6] | (h[7] << 16));
    }
    *reinterpret_cast<uint4*>(D + r * ldd + c) = v;
  }
}

template <typename T>
cudaError_t launch_typed(const float* ws, int slices, int M, int N, long long ldw, float alpha,
                         float beta, T* C, long long ldc, cudaStream_t stream) {
  // (The workspace's cap keeps M * N, and so the CTAs, far below 2^31.)
  const unsigned groups = (unsigned)((N + 127) / 128);
  const unsigned rows = (unsigned)((M + kThreads / 32 - 1) / (kThreads / 32));
  const bool vec = (reinterpret_cast<uintptr_t>(C) & (4 * sizeof(T) - 1)) == 0 && ldc % 4 == 0;
  return launch_gemm_kernel(mx_reduce_kernel<T>, dim3(groups * rows), dim3(kThreads), 0, stream,
                            ws, slices, M, N, ldw, alpha, beta, C, ldc, vec);
}

}  // namespace

cudaError_t launch_mx_align(const void* S, long long rows, int cols, void* D, long long ldd,
                            cudaStream_t stream) {
  const long long ctas = (rows * (ldd / 8) + kThreads - 1) / kThreads;
  return launch_gemm_kernel(mx_align_kernel, dim3((unsigned)(ctas < (1 << 20) ? ctas : 1 << 20)),
                            dim3(kThreads), 0, stream, static_cast<const unsigned short*>(S), rows,
                            cols, static_cast<unsigned short*>(D), ldd);
}

cudaError_t launch_mx_reduce(const float* ws, int slices, int M, int N, long long ldw, float alpha,
                             float beta, void* C, long long ldc, int dtype, cudaStream_t stream) {
  if (dtype == 0)
    return launch_typed(ws, slices, M, N, ldw, alpha, beta, static_cast<float*>(C), ldc, stream);
  if (dtype == 1)
    return launch_typed(ws, slices, M, N, ldw, alpha, beta, static_cast<__half*>(C), ldc, stream);
  return launch_typed(ws, slices, M, N, ldw, alpha, beta, static_cast<__nv_bfloat16*>(C), ldc,
                      stream);
}

}  // namespace dgemm
