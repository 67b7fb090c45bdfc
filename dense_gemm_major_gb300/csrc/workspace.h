// Device workspaces owned by the library: one per (device, stream, use).
#pragma once

#include <cstddef>
#include <mutex>

#include <cuda_runtime_api.h>

#include "dense_gemm.h"

namespace dgemm {

enum WorkspaceUse {
  kWsPartials,   // FP32 partial results: split-K slices, stream-K tiles, ranges of K
  kWsPack,       // copies of operands (transposed, or with aligned rows)
  kWsFlags,      // hand-over flags of cut tiles: zeroed when allocated, then only ever set
                 // to a launch's epoch (or cleared)
  kWsQuantized,  // the quantised X of gemm_mx4_linear
  kWsUses
};

struct StreamEntry;   // a stream's workspaces

// The workspaces of `stream` on the current device, for one call of the
// library.  From the first get() until the object goes, other calls on this
// stream wait when they want a workspace: a host thread's kernels that share
// one are queued together, with none of another thread's between them, and
// nobody replaces a workspace whose address has been taken but not launched
// with.  Calls that need none are not held up.
//
// (cudaStreamPerThread is another stream in each host thread, so each thread
// has its own workspaces for it.)
class StreamWorkspaces {
 public:
  explicit StreamWorkspaces(cudaStream_t stream) noexcept : stream_(stream) {}
  StreamWorkspaces(const StreamWorkspaces&) = delete;
  StreamWorkspaces& operator=(const StreamWorkspaces&) = delete;

  // At least `bytes` of device memory, 256-byte aligned.  A workspace that is
  // too small is replaced by one at least twice its size, and its memory
  // stays allocated until the process exits: work that is queued, and graphs
  // that were captured on this stream, hold its address.  (Doubling bounds
  // what is left behind by the size in use.)
  gemm_status_t get(WorkspaceUse use, size_t bytes, void** out) noexcept;

  // The next epoch of the flags, never 0; after get(kWsFlags).
  unsigned next_epoch() noexcept;

 private:
  cudaStream_t stream_;
  StreamEntry* entry_ = nullptr;
  std::unique_lock<std::mutex> lock_;
};

}  // namespace dgemm
