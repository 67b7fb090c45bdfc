"""Host side of the grouped products' entry points: argument checks and refusals,
none of which needs a GPU."""
import pytest

import __graft_entry__
import dense_gemm_major_gb300 as dg

FAKE = 1 << 40   # 16-byte aligned fake device addresses, never dereferenced
A, B, C, OFF = FAKE, FAKE + (1 << 30), FAKE + (2 << 30), FAKE + (3 << 30)
INVALID, MISALIGNED = dg.GEMM_ERR_INVALID_ARG, dg.GEMM_ERR_MISALIGNED
LARGE = 2 ** 31 - 1023


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()
    return dg.load()


def _product(**kw):
    a = dict(dtype="bf16", op="N", dtype_c="bf16", rows=10, N=32, K=64, groups=3, alpha=1.0, A=A,
             lda=64, B=B, ldb=32, stride_b=64 * 32, off=OFF, beta=0.0, C=C, ldc=32)
    a.update(kw)
    return dg.gemm_grouped(a["dtype"], a["op"], a["dtype_c"], a["rows"], a["N"], a["K"],
                           a["groups"], a["alpha"], a["A"], a["lda"], a["B"], a["ldb"],
                           a["stride_b"], a["off"], a["beta"], a["C"], a["ldc"])


@pytest.mark.parametrize("kw,status", [
    (dict(dtype="f32", dtype_c="f32"), INVALID), (dict(dtype_c="f16"), INVALID),
    (dict(dtype=3), INVALID), (dict(op="C"), INVALID), (dict(rows=-1), INVALID),
    (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(groups=-1), INVALID),
    (dict(groups=1025), INVALID), (dict(rows=LARGE), INVALID), (dict(N=LARGE), INVALID),
    (dict(K=LARGE), INVALID), (dict(A=0), INVALID), (dict(B=0), INVALID), (dict(C=0), INVALID),
    (dict(off=0), INVALID), (dict(lda=63), INVALID), (dict(ldb=31), INVALID),
    (dict(op="T", ldb=63), INVALID), (dict(ldc=31), INVALID), (dict(stride_b=64 * 32 - 8), INVALID),
    (dict(stride_b=-64 * 32), INVALID), (dict(C=A), INVALID), (dict(C=B + 4096), INVALID),
    (dict(C=OFF), INVALID), (dict(C=B + 3 * 64 * 32 * 2 - 2), INVALID),
    (dict(off=OFF + 2), MISALIGNED), (dict(C=C + 1), MISALIGNED),
    (dict(dtype_c="f32", C=C + 2), MISALIGNED), (dict(A=A + 2, lda=72), MISALIGNED),
    (dict(A=A + 1), MISALIGNED), (dict(lda=65), MISALIGNED), (dict(ldb=33, stride_b=4096), MISALIGNED),
    (dict(B=B + 2, stride_b=4096), MISALIGNED), (dict(stride_b=64 * 32 + 4), MISALIGNED),
])
def test_product_refusals(kw, status):
    assert _product(**kw) == status


def _grad(**kw):
    a = dict(dtype="f16", dtype_c="f32", rows=10, M=32, N=64, groups=3, alpha=1.0, A=A, lda=32, X=B,
             ldx=64, off=OFF, beta=0.0, C=C, ldc=64, stride_c=32 * 64)
    a.update(kw)
    return dg.gemm_grouped_grad(a["dtype"], a["dtype_c"], a["rows"], a["M"], a["N"], a["groups"],
                                a["alpha"], a["A"], a["lda"], a["X"], a["ldx"], a["off"],
                                a["beta"], a["C"], a["ldc"], a["stride_c"])


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=0), INVALID), (dict(dtype_c="bf16"), INVALID), (dict(rows=-1), INVALID),
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(groups=-1), INVALID),
    (dict(groups=1025), INVALID), (dict(M=LARGE), INVALID), (dict(N=LARGE), INVALID),
    (dict(rows=LARGE), INVALID), (dict(A=0), INVALID), (dict(X=0), INVALID), (dict(C=0), INVALID),
    (dict(off=0), INVALID), (dict(lda=31), INVALID), (dict(ldx=63), INVALID),
    (dict(ldc=63), INVALID), (dict(stride_c=32 * 64 - 1), INVALID), (dict(stride_c=0), INVALID),
    (dict(C=A), INVALID), (dict(C=B), INVALID), (dict(C=OFF), INVALID),
    (dict(C=A - 3 * 32 * 64 * 4 + 4), INVALID),
    (dict(off=OFF + 1), MISALIGNED), (dict(C=C + 2), MISALIGNED), (dict(lda=36), MISALIGNED),
    (dict(ldx=68), MISALIGNED), (dict(X=B + 1), MISALIGNED), (dict(A=A + 8, lda=40), MISALIGNED),
])
def test_grad_refusals(kw, status):
    assert _grad(**kw) == status


def test_empty_calls_need_no_device():
    assert _product(rows=0, A=0, C=0, off=0) == dg.GEMM_OK
    assert _product(N=0, B=0, C=0) == dg.GEMM_OK
    assert _product(groups=0, B=0, off=0) == dg.GEMM_OK
    assert _product(K=0, A=0, B=0, beta=1.0) == dg.GEMM_OK
    assert _product(alpha=0.0, A=0, B=0, beta=1.0) == dg.GEMM_OK
    assert _grad(M=0, A=0, C=0) == dg.GEMM_OK
    assert _grad(N=0, X=0, C=0) == dg.GEMM_OK
    assert _grad(groups=0, off=0) == dg.GEMM_OK
    assert _grad(rows=0, A=0, X=0, beta=1.0) == dg.GEMM_OK


def test_without_a_gpu_the_calls_say_so():
    """Complete arguments get past the checks (here to the missing device)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake addresses are for machines without a GPU")
    for kw in (dict(), dict(op="T", ldb=64), dict(stride_b=0), dict(groups=1, stride_b=5),
               dict(A=A + 2, K=63, lda=63, ldb=32, stride_b=63 * 32), dict(dtype_c="f32"),
               dict(B=B + 2), dict(N=31, ldb=31, stride_b=64 * 31, ldc=31)):
        assert _product(**kw) == dg.GEMM_ERR_UNSUPPORTED_DEVICE, kw
    for kw in (dict(), dict(groups=1, stride_c=0), dict(M=31, lda=31, A=A + 2), dict(rows=0, A=0),
               dict(dtype_c="f16", C=C + 2)):
        assert _grad(**kw) == dg.GEMM_ERR_UNSUPPORTED_DEVICE, kw
