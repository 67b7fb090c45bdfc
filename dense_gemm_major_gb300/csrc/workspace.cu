// The library's device workspaces.  See workspace.h.
#include "workspace.h"

#include <map>
#include <mutex>
#include <tuple>

namespace dgemm {
namespace {

struct Workspace {
  void* ptr = nullptr;
  size_t bytes = 0;
  unsigned epoch = 0;   // kWsFlags: the last epoch handed to a launch
};

std::mutex g_mu;
std::map<std::tuple<int, cudaStream_t, int>, Workspace> g_workspaces;   // guarded by g_mu

gemm_status_t grow(Workspace& w, WorkspaceUse use, size_t bytes, cudaStream_t stream) {
  size_t size = bytes > 2 * w.bytes ? bytes : 2 * w.bytes;
  void* p = nullptr;
  if (cudaMalloc(&p, size) != cudaSuccess) {
    cudaGetLastError();
    size = bytes;
    if (cudaMalloc(&p, size) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_LAUNCH;
    }
  }
  if (use == kWsFlags && cudaMemsetAsync(p, 0, size, stream) != cudaSuccess) {
    cudaGetLastError();
    cudaFree(p);
    return GEMM_ERR_LAUNCH;
  }
  w.ptr = p;
  w.bytes = size;
  return GEMM_OK;
}

}  // namespace

gemm_status_t get_workspace(cudaStream_t stream, WorkspaceUse use, size_t bytes,
                            void** out) noexcept try {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return GEMM_ERR_UNSUPPORTED_DEVICE;
  }
  std::lock_guard<std::mutex> lock(g_mu);
  Workspace& w = g_workspaces[std::make_tuple(dev, stream, (int)use)];
  if (w.bytes < bytes) {
    const gemm_status_t st = grow(w, use, bytes, stream);
    if (st != GEMM_OK) return st;
  }
  *out = w.ptr;
  return GEMM_OK;
} catch (...) {   // no host memory
  return GEMM_ERR_LAUNCH;
}

unsigned next_epoch(cudaStream_t stream) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) cudaGetLastError();
  std::lock_guard<std::mutex> lock(g_mu);
  Workspace& w = g_workspaces[std::make_tuple(dev, stream, (int)kWsFlags)];
  if (++w.epoch == 0) w.epoch = 1;
  return w.epoch;
}

}  // namespace dgemm
