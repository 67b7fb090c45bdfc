"""The torch wrappers of the grouped products and of those with 4-bit weights let other
Python threads run while the library's call is under way.  On the CPU, in a process of its
own: the extension beside a stand-in for the library whose calls take half a second."""
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
int gemm_grouped(...) { return busy(); }
int gemm_grouped_grad(...) { return busy(); }
int gemm_q4_linear(...) { return busy(); }
}
"""

SCRIPT = r"""
import importlib.util, sys, threading, time, types

spec = importlib.util.spec_from_file_location("_groupcall", sys.argv[1])
ext = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ext)
device = types.SimpleNamespace(index=0)

class Tensor:
    is_cuda = True
    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.device = shape, dtype, device
    def stride(self):
        steps, step = [], 1
        for n in reversed(self.shape):
            steps.insert(0, step)
            step *= n
        return tuple(steps)
    def data_ptr(self):
        return 1 << 20

class Weights:
    codes, _scales, _zeros = (Tensor((8, 32), "uint8"), Tensor((2, 8), "bfloat16"), None)
    experts, rows, cols, group, _ld = 0, 8, 64, 32, 32

def empty(size, dtype=None, device=None):
    return Tensor(size, dtype)

torch = types.SimpleNamespace(
    float32="float32", float16="float16", bfloat16="bfloat16", uint8="uint8", int32="int32",
    empty=empty,
    _C=types.SimpleNamespace(_cuda_getCurrentRawStream=lambda i: 0, _cuda_getDevice=lambda: 0))
ext.setup(torch, Weights, RuntimeError)
x, w, off = Tensor((8, 64), "bfloat16"), Tensor((2, 64, 16), "bfloat16"), Tensor((3,), "int32")
calls = {"grouped_matmul": (x, w, off, None, None, 1.0, 0.0, None),
         "grouped_grad": (x, x, off, None, None, 1.0, 0.0, None),
         "q4_linear": (x, Weights(), None, None, None)}
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
    ext = shutil.copy(_build.GROUP_EXT, d)
    out = subprocess.run([sys.executable, str(d / "script.py"), ext], check=True, timeout=60,
                         stdout=subprocess.PIPE, cwd=d, text=True,
                         env={k: v for k, v in os.environ.items() if k != "LD_LIBRARY_PATH"})
    return {line.split()[0]: float(line.split()[1]) for line in out.stdout.splitlines()}


@pytest.mark.parametrize("name", ["grouped_matmul", "grouped_grad", "q4_linear"])
def test_other_threads_run_during_a_call(pauses, name):
    assert pauses[name] < 0.4
