// Device workspaces owned by the library: one per (device, stream, use).
#pragma once

#include <cstddef>
#include <cuda_runtime_api.h>

#include "dense_gemm.h"

namespace dgemm {

enum WorkspaceUse {
  kWsPartials,   // FP32 partial results: split-K slices, stream-K tiles, ranges of K
  kWsPack,       // copies of FP32 operands (transposed, or with aligned rows)
  kWsFlags,      // hand-over flags of cut tiles: zeroed when allocated, then only ever set
                 // to a launch's epoch (or cleared)
  kWsQuantized,  // the quantised X of gemm_mx4_linear
};

// At least `bytes` of device memory for work queued on `stream`, 256-byte
// aligned.  A workspace that is too small is replaced by one at least twice
// its size, and its memory stays allocated until the process exits: work
// that is queued, and graphs that were captured on this stream, hold its
// address.  (Doubling bounds what is left behind by the size in use.)
// Throws nothing.
gemm_status_t get_workspace(cudaStream_t stream, WorkspaceUse use, size_t bytes,
                            void** out) noexcept;

// The next epoch of the flags of (current device, stream); never 0.
unsigned next_epoch(cudaStream_t stream);

}  // namespace dgemm
