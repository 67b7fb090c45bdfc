"""The torch wrappers of the microscaled operators let other Python threads run
while the library's call is under way.  On the CPU, in a process of its own: the
extension beside a stand-in for the library whose calls take half a second."""
import os
import shutil
import subprocess
import sys

import pytest

import __graft_entry__
from dense_gemm_major_gb300 import _build

LIBRARY = r"""
#include <unistd.h>
extern "C" {
static int busy() { usleep(500000); return 0; }
int gemm_mx_code_ld(int, int) { return 64; }
long long gemm_mx_scale_bytes(int, int) { return 512; }
int gemm_mx_quantize(...) { return busy(); }
int gemm_mx_dequantize(...) { return busy(); }
int gemm_mx4(...) { return busy(); }
int gemm_mx4_linear(...) { return busy(); }
int gemm_mx_grad(...) { return busy(); }
}
"""

SCRIPT = r"""
import importlib.util, sys, threading, time, types

spec = importlib.util.spec_from_file_location("_mxcall", sys.argv[1])
ext = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ext)
device = types.SimpleNamespace(index=0)

class Tensor:
    is_cuda = True
    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.device = shape, dtype, device
    def stride(self):
        return (self.shape[-1], 1)[-len(self.shape):]
    def data_ptr(self):
        return 1 << 20
    def is_contiguous(self):
        return True
    def numel(self):
        return 1 << 20

class Quantized:
    def __init__(self, rows):
        self.rows, self.cols, self.fmt, self._ld, self._buffer = rows, 64, "mxfp4", 32, None
        self._codes, self._scales = Tensor((rows, 32), "uint8"), Tensor((512,), "uint8")
        self._device = device

def empty(size, dtype=None, device=None):
    return Tensor(size if isinstance(size, tuple) else (size,), dtype)

torch = types.SimpleNamespace(
    float32="float32", float16="float16", bfloat16="bfloat16", uint8="uint8", empty=empty,
    _C=types.SimpleNamespace(_cuda_getCurrentRawStream=lambda i: 0, _cuda_getDevice=lambda: 0))
ext.setup(torch, Quantized, RuntimeError)
x, q = Tensor((8, 64), "bfloat16"), Quantized(8)
calls = {"quantize": (x, "mxfp4", None), "dequantize": (q, None, None, None),
         "matmul": (q, q, None, None, 1.0, 0.0, None), "linear": (x, q, None, None),
         "grad": (Tensor((4, 8), "bfloat16"), q, None, None, 1.0, 0.0, None)}
for name, args in calls.items():
    thread = threading.Thread(target=getattr(ext, name), args=args)
    worst, last = 0.0, time.monotonic()
    thread.start()
    while thread.is_alive():
        time.sleep(0.01)
        now = time.monotonic()
        worst, last = max(worst, now - last), now
    print(name, round(worst, 3))
"""


@pytest.fixture(scope="module")
def pauses(tmp_path_factory):
    """The longest time that the main thread stood still, for each function."""
    __graft_entry__.build()
    d = tmp_path_factory.mktemp("threads")
    (d / "library.cpp").write_text(LIBRARY)
    (d / "script.py").write_text(SCRIPT)
    subprocess.check_call(["g++", "-fPIC", "-shared", str(d / "library.cpp"), "-o",
                           str(d / "libdense_gemm.so")])
    ext = shutil.copy(_build.EXT, d)
    out = subprocess.run([sys.executable, str(d / "script.py"), ext], check=True, timeout=60,
                         stdout=subprocess.PIPE, cwd=d, text=True,
                         env={k: v for k, v in os.environ.items() if k != "LD_LIBRARY_PATH"})
    return {line.split()[0]: float(line.split()[1]) for line in out.stdout.splitlines()}


@pytest.mark.parametrize("name", ["quantize", "dequantize", "matmul", "linear", "grad"])
def test_other_threads_run_during_a_call(pauses, name):
    assert pauses[name] < 0.4
