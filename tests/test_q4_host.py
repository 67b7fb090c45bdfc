"""Host side of the entry point for 4-bit weights: argument checks and refusals, none
of which needs a GPU."""
import pytest

import __graft_entry__
import dense_gemm_major_gb300 as dg

FAKE = 1 << 40   # 16-byte aligned fake device addresses, never dereferenced
X, Q, S, Z, OFF, Y = (FAKE + (i << 30) for i in range(6))
INVALID, MISALIGNED = dg.GEMM_ERR_INVALID_ARG, dg.GEMM_ERR_MISALIGNED
LARGE = 2 ** 31 - 1023


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()
    return dg.load()


def _call(**kw):
    a = dict(dtype="bf16", group=64, rows=4, N=48, K=160, experts=0, X=X, ldx=160, q=Q, ldq=80, s=S,
             z=Z, off=0, Y=Y, ldy=48)
    a.update(kw)
    return dg.gemm_q4_linear(a["dtype"], a["group"], a["rows"], a["N"], a["K"], a["experts"],
                             a["X"], a["ldx"], a["q"], a["ldq"], a["s"], a["z"], a["off"], a["Y"],
                             a["ldy"])


@pytest.mark.parametrize("kw,status", [
    (dict(dtype="f32"), INVALID), (dict(dtype=3), INVALID), (dict(group=0), INVALID),
    (dict(group=48), INVALID), (dict(group=-32), INVALID), (dict(rows=-1), INVALID),
    (dict(N=-1), INVALID), (dict(K=-1), INVALID), (dict(experts=-1), INVALID),
    (dict(experts=1025, off=OFF), INVALID), (dict(rows=LARGE), INVALID), (dict(N=LARGE), INVALID),
    (dict(K=LARGE), INVALID), (dict(experts=2), INVALID), (dict(off=OFF), INVALID),
    (dict(X=0), INVALID), (dict(q=0), INVALID), (dict(s=0), INVALID), (dict(Y=0), INVALID),
    (dict(ldx=159), INVALID), (dict(ldq=64), INVALID), (dict(ldy=47), INVALID),
    (dict(Y=X), INVALID), (dict(Y=Q + 47 * 80 + 78), INVALID), (dict(Y=S), INVALID),
    (dict(Y=Z + 142), INVALID), (dict(experts=2, off=OFF, Y=OFF), INVALID),
    (dict(experts=2, off=OFF, Y=S + 2 * 48 * 3 * 2 - 2), INVALID),
    (dict(q=Q + 8), MISALIGNED), (dict(ldq=88), MISALIGNED), (dict(s=S + 1), MISALIGNED),
    (dict(Y=Y + 1), MISALIGNED), (dict(experts=2, off=OFF + 2), MISALIGNED),
    (dict(X=X + 1), MISALIGNED), (dict(ldx=161), MISALIGNED), (dict(X=X + 2, ldx=168), MISALIGNED),
])
def test_refusals(kw, status):
    assert _call(**kw) == status


@pytest.mark.parametrize("kw", [
    dict(Y=S + 48 * 2 - 2), dict(Y=Z + 46), dict(K=64, ldx=64, Y=S + 48 * 2 - 2),
    dict(experts=3, off=OFF, Y=S + 3 * 48 * 2 - 2), dict(experts=3, off=OFF, Y=Z + 3 * 48 - 2)])
def test_overlaps_with_scales_of_the_largest_group(kw):
    """K + group - 1 is past 2^31 - 1: there is still one group to a row."""
    assert _call(group=2 ** 31 - 32, **kw) == INVALID


def test_empty_calls_need_no_device():
    assert _call(rows=0, X=0, Y=0) == dg.GEMM_OK
    assert _call(N=0, q=0, s=0, Y=0) == dg.GEMM_OK
    assert _call(experts=2, off=OFF, rows=0) == dg.GEMM_OK


def test_without_a_gpu_the_calls_say_so():
    """Complete arguments get past the checks (here to the missing device)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake addresses are for machines without a GPU")
    for kw in (dict(), dict(z=0), dict(experts=3, off=OFF), dict(K=159, ldx=159, X=X + 2),
               dict(group=1 << 20), dict(Y=Y + 2, ldy=49), dict(K=0, X=0, q=0, s=0),
               dict(rows=5000), dict(Y=S + 48 * 3 * 2)):
        assert _call(**kw) == dg.GEMM_ERR_UNSUPPORTED_DEVICE, kw
