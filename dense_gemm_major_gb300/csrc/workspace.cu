// The library's device workspaces.  See workspace.h.
#include "workspace.h"

#include <atomic>
#include <map>
#include <tuple>

namespace dgemm {

struct Workspace {
  void* ptr = nullptr;
  size_t bytes = 0;
};

struct StreamEntry {
  std::mutex mu;
  Workspace ws[kWsUses];   // guarded by mu
  unsigned epoch = 0;      // the last one handed to a launch; guarded by mu
};

namespace {

// Device, stream, and for cudaStreamPerThread the host thread.  Entries stay
// for good.
using Key = std::tuple<int, cudaStream_t, unsigned long long>;

StreamEntry* entry_of(int dev, cudaStream_t stream) {
  static std::mutex mu;
  static auto* entries = new std::map<Key, StreamEntry>;   // guarded by mu
  static std::atomic<unsigned long long> threads{0};
  static thread_local const unsigned long long thread = ++threads;
  std::lock_guard<std::mutex> lock(mu);
  return &(*entries)[Key(dev, stream, stream == cudaStreamPerThread ? thread : 0)];
}

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

gemm_status_t StreamWorkspaces::get(WorkspaceUse use, size_t bytes, void** out) noexcept try {
  if (entry_ == nullptr) {
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) {
      cudaGetLastError();
      return GEMM_ERR_UNSUPPORTED_DEVICE;
    }
    StreamEntry* entry = entry_of(dev, stream_);
    lock_ = std::unique_lock<std::mutex>(entry->mu);
    entry_ = entry;
  }
  Workspace& w = entry_->ws[use];
  if (w.bytes < bytes) {
    const gemm_status_t st = grow(w, use, bytes, stream_);
    if (st != GEMM_OK) return st;
  }
  *out = w.ptr;
  return GEMM_OK;
} catch (...) {   // no host memory
  return GEMM_ERR_LAUNCH;
}

unsigned StreamWorkspaces::next_epoch() noexcept {
  if (++entry_->epoch == 0) entry_->epoch = 1;
  return entry_->epoch;
}

}  // namespace dgemm
