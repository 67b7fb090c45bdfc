"""The library's workspaces (csrc/workspace.cu) on the CPU: compiled by the
host compiler against a stand-in for the few CUDA runtime calls they make,
which hands out addresses and records what is freed."""
import ctypes
import os
import subprocess
import threading

import pytest

from dense_gemm_major_gb300 import _build

PARTIALS, PACK, FLAGS, QUANTIZED = range(4)

HARNESS = r"""
#include "workspace.cu"
#include <cstdint>
#include <vector>

static uintptr_t g_next = 1 << 20;
static size_t g_limit = (size_t)1 << 40;
static std::vector<void*> g_freed;
static std::vector<size_t> g_sizes, g_cleared;

extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = 0; return cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaMalloc(void** p, size_t n) {
  if (n > g_limit) return cudaErrorMemoryAllocation;
  *p = (void*)g_next;
  g_next += (n + 4095) / 4096 * 4096;
  g_sizes.push_back(n);
  return cudaSuccess;
}
cudaError_t cudaFree(void* p) { g_freed.push_back(p); return cudaSuccess; }
cudaError_t cudaMemsetAsync(void*, int, size_t n, cudaStream_t) {
  g_cleared.push_back(n);
  return cudaSuccess;
}
void t_limit(size_t n) { g_limit = n; }
int t_freed() { return (int)g_freed.size(); }
int t_allocations() { return (int)g_sizes.size(); }
size_t t_size(int i) { return g_sizes[i]; }
size_t t_cleared() { size_t s = 0; for (size_t n : g_cleared) s += n; return s; }
void* t_open(uintptr_t stream) { return new dgemm::StreamWorkspaces((cudaStream_t)stream); }
void* t_use(void* w, int use, size_t bytes) {
  void* p = nullptr;
  return ((dgemm::StreamWorkspaces*)w)->get((dgemm::WorkspaceUse)use, bytes, &p) == GEMM_OK
             ? p : nullptr;
}
unsigned t_epoch(void* w) { return ((dgemm::StreamWorkspaces*)w)->next_epoch(); }
void t_close(void* w) { delete (dgemm::StreamWorkspaces*)w; }
void* t_get(uintptr_t stream, int use, size_t bytes) {   // a call that needs one workspace
  dgemm::StreamWorkspaces w((cudaStream_t)stream);
  void* p = nullptr;
  return w.get((dgemm::WorkspaceUse)use, bytes, &p) == GEMM_OK ? p : nullptr;
}
}
"""


@pytest.fixture
def ws(tmp_path):
    """A fresh copy of the workspaces with nothing allocated."""
    src, lib = tmp_path / "harness.cpp", tmp_path / "harness.so"
    src.write_text(HARNESS)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_build.nvcc())) or "/usr/local/cuda",
                        "include")
    # (-Bsymbolic: the stand-in's calls, even where torch has loaded the real ones.)
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-fPIC", "-shared", "-pthread",
                           "-Wl,-Bsymbolic", str(src), "-o", str(lib), "-I", _build.CSRC, "-I", _build.INCLUDE, "-I", cuda])
    h = ctypes.CDLL(str(lib))
    h.t_get.restype = ctypes.c_void_p
    h.t_get.argtypes = [ctypes.c_size_t, ctypes.c_int, ctypes.c_size_t]
    h.t_size.restype = h.t_cleared.restype = ctypes.c_size_t
    h.t_open.restype = h.t_use.restype = ctypes.c_void_p
    h.t_open.argtypes = [ctypes.c_size_t]
    h.t_use.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t]
    h.t_close.argtypes = h.t_epoch.argtypes = [ctypes.c_void_p]
    h.t_limit.argtypes = [ctypes.c_size_t]
    return h


def test_growth_keeps_the_outgrown_memory(ws):
    """A graph captured with the first address stays valid: nothing is freed,
    and doubling keeps the number of allocations small."""
    first = ws.t_get(16, QUANTIZED, 1000)
    assert ws.t_get(16, QUANTIZED, 400) == first
    second = ws.t_get(16, QUANTIZED, 1001)
    assert second != first and ws.t_size(1) == 2000
    assert ws.t_get(16, QUANTIZED, 2000) == second
    for n in range(2001, 60000, 1):
        ws.t_get(16, QUANTIZED, n)
    assert ws.t_freed() == 0 and ws.t_allocations() <= 7


VALUES = 4


@pytest.mark.parametrize("needs", [(200, 250), (1, 200, 250, 256), (130, 131, 255), (256, 3),
                                   tuple(range(1, 257)), (100, 300)])
def test_the_weights_workspace_keeps_its_bound(ws, needs):
    """MB that calls need one after the other: no workspace for 4-bit weights in 16 bits is
    above 256 MB as long as no call needs more, and those that were outgrown are together
    smaller than the one in use."""
    for n in needs:
        assert ws.t_get(16, VALUES, n << 20) is not None
    sizes = [ws.t_size(i) for i in range(ws.t_allocations())]
    assert max(needs) << 20 <= sizes[-1] <= (256 << 20 if max(needs) <= 256 else 512 << 20)
    assert sum(sizes[:-1]) < sizes[-1] and ws.t_freed() == 0


def test_little_memory_for_the_weights_workspace(ws):
    """The power of two does not fit: what the call needs."""
    ws.t_limit(200 << 20)
    assert ws.t_get(16, VALUES, 190 << 20) is not None and ws.t_size(0) == 190 << 20


def test_streams_and_uses_do_not_share(ws):
    got = {ws.t_get(s, use, 4096) for s in (0, 16, 32) for use in (PARTIALS, PACK, FLAGS, QUANTIZED)}
    assert len(got) == 12 and None not in got


def test_flags_are_cleared_whole_when_allocated(ws):
    ws.t_get(16, FLAGS, 100)
    ws.t_get(16, FLAGS, 101)
    ws.t_get(16, FLAGS, 200)
    assert ws.t_cleared() == 100 + 200
    ws.t_get(16, PARTIALS, 5000)
    assert ws.t_cleared() == 300


def test_little_memory(ws):
    """Twice the size does not fit: what the call needs; that neither: an
    error, and the workspace stays as it was."""
    first = ws.t_get(16, PACK, 1000)
    ws.t_limit(1500)
    second = ws.t_get(16, PACK, 1200)
    assert second not in (None, first) and ws.t_size(1) == 1200
    assert ws.t_get(16, PACK, 1600) is None
    assert ws.t_get(16, PACK, 1200) == second


def _in_thread(f):
    """f() started in a thread of its own; (thread, its results)."""
    out = []
    t = threading.Thread(target=lambda: out.append(f()), daemon=True)
    t.start()
    return t, out


@pytest.mark.parametrize("first,second", [(QUANTIZED, QUANTIZED), (QUANTIZED, PARTIALS)])
def test_a_call_keeps_others_on_its_stream_waiting(ws, first, second):
    """From a call's first workspace until its last kernel is queued no other
    thread gets one of the stream, be it to write it or to replace it."""
    call = ws.t_open(16)
    mine = ws.t_use(call, first, 1000)
    t, out = _in_thread(lambda: ws.t_get(16, second, 5000))
    t.join(0.2)
    assert t.is_alive() and ws.t_allocations() == 1
    assert ws.t_use(call, first, 500) == mine
    # Another stream, and a call that needs no workspace, go on.
    other, got = _in_thread(lambda: ws.t_get(32, first, 1000))
    other.join(20)
    assert got and got[0] is not None
    ws.t_close(ws.t_open(16))
    ws.t_close(call)
    t.join(20)
    assert out and out[0] not in (None, mine)


def test_epochs_are_never_repeated(ws):
    seen = []
    for _ in range(3):
        call = ws.t_open(16)
        ws.t_use(call, FLAGS, 64)
        seen += [ws.t_epoch(call), ws.t_epoch(call)]
        ws.t_close(call)
    assert seen == [1, 2, 3, 4, 5, 6]


def test_the_per_thread_stream_is_another_one_in_each_thread(ws):
    per_thread = 2   # cudaStreamPerThread
    here = ws.t_get(per_thread, QUANTIZED, 1000)
    t, out = _in_thread(lambda: ws.t_get(per_thread, QUANTIZED, 1000))
    t.join(20)
    assert out[0] not in (None, here)
    assert ws.t_get(per_thread, QUANTIZED, 1000) == here
