// The sum of the FP32 partial results of a product split along K, with its
// epilogue: C := alpha * sum + beta * C, slices added in order.  The partial
// results have just been written and are read from L2.
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
