"""Host side of the microscaled entry points: sizes, argument checks and
refusals (no GPU needed), and the plain implementation the GPU tests use,
checked against the format's definition by hand."""
import numpy as np
import pytest

import __graft_entry__
import dense_gemm_major_gb300 as dg
import mx_reference as ref

FAKE = 1 << 40   # 16-byte aligned fake device addresses, never dereferenced
Q, S, X, Y = FAKE, FAKE + (1 << 30), FAKE + (2 << 30), FAKE + (3 << 30)
Q2, S2 = FAKE + (4 << 30), FAKE + (5 << 30)
INVALID, MISALIGNED = dg.GEMM_ERR_INVALID_ARG, dg.GEMM_ERR_MISALIGNED


@pytest.fixture(scope="module", autouse=True)
def built():
    __graft_entry__.build()
    return dg.load()


@pytest.mark.parametrize("K,fp4,int8", [(0, 0, 0), (1, 16, 16), (16, 16, 16), (17, 16, 32),
                                        (32, 16, 32), (33, 32, 48), (777, 400, 784)])
def test_code_pitch(K, fp4, int8):
    assert dg.gemm_mx_code_ld("mxfp4", K) == fp4
    assert dg.gemm_mx_code_ld("mxint8", K) == int8


@pytest.mark.parametrize("R,K,tiles", [(0, 5, 0), (5, 0, 0), (1, 1, 1), (128, 128, 1),
                                       (129, 128, 2), (128, 129, 2), (1000, 777, 56),
                                       (2 ** 20, 2 ** 20, 2 ** 26)])
def test_scale_bytes(R, K, tiles):
    assert dg.gemm_mx_scale_bytes(R, K) == 512 * tiles


def test_bad_sizes():
    assert dg.gemm_mx_code_ld("mxfp4", -1) == -1
    assert dg.gemm_mx_code_ld("mxfp6", 32) == -1
    assert dg.gemm_mx_scale_bytes(-1, 4) == -1 and dg.gemm_mx_scale_bytes(4, -1) == -1


def _quantize(fmt="mxfp4", dtype="bf16", op="N", R=4, K=64, X=X, ldx=64, q=Q, ldq=64, s=S):
    return dg.gemm_mx_quantize(fmt, dtype, op, R, K, X, ldx, q, ldq, s)


@pytest.mark.parametrize("kw,status", [
    (dict(fmt="mxfp6"), INVALID), (dict(dtype=3), INVALID), (dict(op="C"), INVALID),
    (dict(R=-1), INVALID), (dict(K=-1), INVALID), (dict(X=0), INVALID), (dict(q=0), INVALID),
    (dict(s=0), INVALID), (dict(ldx=63), INVALID), (dict(op="T", ldx=3), INVALID),
    (dict(ldq=16), INVALID), (dict(fmt="mxint8", ldq=48), INVALID),
    (dict(ldq=40), MISALIGNED), (dict(q=Q + 8), MISALIGNED), (dict(s=S + 4), MISALIGNED),
    (dict(X=X + 1), MISALIGNED), (dict(dtype="f32", X=X + 2), MISALIGNED),
    (dict(q=X), INVALID), (dict(s=X + 256), INVALID), (dict(s=Q + 64), INVALID),
])
def test_quantize_refusals(kw, status):
    assert _quantize(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=7), INVALID), (dict(dtype=-1), INVALID), (dict(R=-1), INVALID),
    (dict(K=-1), INVALID), (dict(Y=0), INVALID), (dict(ldy=63), INVALID), (dict(q=0), INVALID),
    (dict(s=0), INVALID), (dict(ldq=16), INVALID), (dict(ldq=33), MISALIGNED),
    (dict(q=Q + 1), MISALIGNED), (dict(s=S + 8), MISALIGNED), (dict(Y=Y + 1), MISALIGNED),
    (dict(Y=Q), INVALID), (dict(Y=S), INVALID),
])
def test_dequantize_refusals(kw, status):
    a = dict(fmt="mxfp4", dtype="f16", R=4, K=64, q=Q, ldq=32, s=S, Y=Y, ldy=64)
    a.update(kw)
    assert dg.gemm_mx_dequantize(a["fmt"], a["dtype"], a["R"], a["K"], a["q"], a["ldq"], a["s"],
                                 a["Y"], a["ldy"]) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), INVALID), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-1), INVALID),
    (dict(a=0), INVALID), (dict(sa=0), INVALID), (dict(b=0), INVALID), (dict(sb=0), INVALID),
    (dict(C=0), INVALID), (dict(ldc=7), INVALID), (dict(lda=16), INVALID), (dict(ldb=16), INVALID),
    (dict(lda=36), MISALIGNED), (dict(b=Q2 + 2), MISALIGNED), (dict(sb=S2 + 1), MISALIGNED),
    (dict(C=Y + 1), MISALIGNED), (dict(C=Q), INVALID), (dict(C=S2), INVALID),
])
def test_product_refusals(kw, status):
    a = dict(dtype="bf16", M=4, N=8, K=64, a=Q, lda=32, sa=S, b=Q2, ldb=32, sb=S2, C=Y, ldc=8)
    a.update(kw)
    assert dg.gemm_mx4(a["dtype"], a["M"], a["N"], a["K"], 1.0, a["a"], a["lda"], a["sa"], a["b"],
                       a["ldb"], a["sb"], 0.0, a["C"], a["ldc"]) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=3), INVALID), (dict(M=-1), INVALID), (dict(X=0), INVALID), (dict(ldx=63), INVALID),
    (dict(w=0), INVALID), (dict(sw=0), INVALID), (dict(Y=0), INVALID), (dict(ldy=7), INVALID),
    (dict(ldw=8), INVALID), (dict(w=Q + 8), MISALIGNED), (dict(X=X + 1), MISALIGNED),
    (dict(Y=X), INVALID), (dict(Y=Q), INVALID),
])
def test_linear_refusals(kw, status):
    a = dict(dtype="f16", M=4, N=8, K=64, X=X, ldx=64, w=Q, ldw=32, sw=S, Y=Y, ldy=8)
    a.update(kw)
    assert dg.gemm_mx4_linear(a["dtype"], a["M"], a["N"], a["K"], a["X"], a["ldx"], a["w"],
                              a["ldw"], a["sw"], a["Y"], a["ldy"]) == status


@pytest.mark.parametrize("kw,status", [
    (dict(fmt=2), INVALID), (dict(dtype="f32", dtype_c="f32"), INVALID),
    (dict(dtype_c="f16"), INVALID), (dict(op=5), INVALID), (dict(M=-1), INVALID),
    (dict(A=0), INVALID), (dict(lda=63), INVALID), (dict(op="T", lda=3), INVALID),
    (dict(b=0), INVALID), (dict(sb=0), INVALID), (dict(ldb=0), INVALID), (dict(C=0), INVALID),
    (dict(ldc=7), INVALID), (dict(lda=65), MISALIGNED), (dict(A=X + 2), MISALIGNED),
    (dict(b=Q + 4), MISALIGNED), (dict(sb=S + 4), MISALIGNED), (dict(C=Y + 1), MISALIGNED),
    (dict(C=X), INVALID), (dict(C=Q), INVALID), (dict(C=S), INVALID),
])
def test_grad_refusals(kw, status):
    a = dict(fmt="mxint8", dtype="bf16", op="N", dtype_c="bf16", M=4, N=8, K=64, A=X, lda=64, b=Q,
             ldb=16, sb=S, C=Y, ldc=8)
    a.update(kw)
    assert dg.gemm_mx_grad(a["fmt"], a["dtype"], a["op"], a["dtype_c"], a["M"], a["N"], a["K"],
                           1.0, a["A"], a["lda"], a["b"], a["ldb"], a["sb"], 0.0, a["C"],
                           a["ldc"]) == status


def test_empty_calls_need_no_device():
    assert _quantize(R=0, X=0, q=0, s=0) == dg.GEMM_OK
    assert _quantize(K=0, X=0, q=0, s=0) == dg.GEMM_OK
    assert dg.gemm_mx_dequantize("mxint8", "f32", 0, 9, 0, 0, 0, 0, 0) == dg.GEMM_OK
    assert dg.gemm_mx4("f32", 0, 5, 64, 1.0, 0, 0, 0, 0, 0, 0, 0.0, 0, 5) == dg.GEMM_OK
    assert dg.gemm_mx4_linear("f16", 5, 0, 64, 0, 0, 0, 0, 0, 0, 0) == dg.GEMM_OK
    assert dg.gemm_mx_grad("mxfp4", "f16", "T", "f32", 0, 5, 64, 1.0, 0, 0, 0, 0, 0, 0.0, 0,
                           5) == dg.GEMM_OK


def test_valid_calls_without_a_gpu_fail_loudly():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    st = dg.GEMM_ERR_UNSUPPORTED_DEVICE
    assert _quantize() == st
    assert dg.gemm_mx4("f32", 4, 8, 64, 1.0, Q, 32, S, Q2, 32, S2, 0.0, Y, 8) == st
    assert dg.gemm_mx4("f32", 4, 8, 0, 1.0, 0, 0, 0, 0, 0, 0, 0.0, Y, 8) == st


@pytest.mark.parametrize("op,M,K,lda,A,misaligned", [
    ("N", 4, 63, 63, X, False), ("N", 4, 63, 63, X + 2, False), ("N", 4, 63, 63, X + 1, True),
    ("T", 4, 64, 4, X + 2, False), ("T", 5, 64, 5, X, False), ("N", 4, 63, 65, X, True),
    ("N", 4, 64, 64, X + 2, True), ("T", 8, 64, 8, X + 2, True), ("T", 4, 64, 5, X, True),
])
def test_grad_takes_packed_operands_of_any_width(op, M, K, lda, A, misaligned):
    import torch
    if not misaligned and torch.cuda.is_available():
        pytest.skip("a GPU is present")
    st = dg.gemm_mx_grad("mxint8", "bf16", op, "bf16", M, 8, K, 1.0, A, lda, Q, 16, S, 0.0, Y, 8)
    assert st == (MISALIGNED if misaligned else dg.GEMM_ERR_UNSUPPORTED_DEVICE)


def test_extension_is_named_for_its_interpreter():
    import sysconfig

    from dense_gemm_major_gb300 import _build
    assert _build.EXT.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert dg._load_mx().__file__ == _build.EXT


def test_wrappers_refuse_wrong_tensors():
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        dg.mx_quantize(x)
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    q = dg.MXTensor(codes, scales, 64)
    assert q.shape == (4, 64)
    for bad in [lambda: dg.MXTensor(codes, scales, 65), lambda: dg.MXTensor(codes, scales, 33, "f4"),
                lambda: dg.MXTensor(codes, scales[:500], 64),
                lambda: dg.MXTensor(codes.t(), scales, 4),
                lambda: dg.MXTensor(codes, scales, 33, "mxint8"),
                lambda: dg.mx_matmul(q, q), lambda: dg.mx_linear(x, q), lambda: dg.mx_grad(x, q),
                lambda: dg.mx_dequantize(q)]:
        with pytest.raises(ValueError):
            bad()


# ------------------------------------------------------------ the plain implementation

def test_reference_rounds_to_the_nearest_code_and_ties_to_even():
    # amax 4 makes the scale 2^(2-2) = 1.
    x = np.array([[4.0, 0.25, 0.250001, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.000001, 7.9, -0.25, -0.75,
                   -6.0] + [0.0] * 18])
    c, s = ref.quantize(x, "mxfp4")
    assert s.tolist() == [[127]]
    assert (c[0, :14] & 7).tolist() == [6, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 0, 2, 7]
    v = ref.values(c, s, "mxfp4")
    assert v[0, :3].tolist() == [4.0, 0.0, 0.5] and v[0, 13] == -6.0


def test_reference_int8_and_special_blocks():
    x = np.zeros((1, 160))
    x[0, :4] = [1.0, 0.5 / 64, 1.5 / 64, -127.6 / 64]   # amax in [1, 2): scale 1
    x[0, 32] = np.inf
    x[0, 64] = np.nan
    x[0, 96] = 2.0 ** -149
    c, s = ref.quantize(x, "mxint8")
    assert s[0].tolist() == [127, 255, 255, 0, 0]
    assert c[0, :4].tolist() == [64, 0, 2, -127]
    v = ref.values(c, s, "mxint8")
    assert np.isnan(v[0, 32:96]).all() and not v[0, 96:].any()


@pytest.mark.parametrize("fmt", ["mxfp4", "mxint8"])
def test_reference_pack_round_trip(fmt):
    rng = np.random.default_rng(1)
    c, s = ref.quantize(rng.standard_normal((130, 77)), fmt)
    c2, s2 = ref.unpack(*ref.pack(c, s, fmt), 77, fmt)
    assert (c2 == c).all() and (s2 == s).all()
    v = ref.values(c, s, fmt)
    again = ref.quantize(v, fmt)
    assert (ref.values(*again, fmt) == v).all()


class FakeTensor:
    """What the wrappers read of a tensor that claims to be on a GPU."""
    is_cuda = True

    def __init__(self, shape, dtype, device, address=FAKE):
        import torch
        self.shape, self.dtype, self.device = shape, dtype, torch.device(device)
        self.address = address

    def stride(self):
        return (self.shape[-1], 1)[-len(self.shape):]

    def data_ptr(self):
        return self.address

    def is_contiguous(self):
        return True

    def numel(self):
        return int(np.prod(self.shape))


def _fake_quantized(device, rows=8, cols=64, fmt="mxfp4"):
    import torch
    width = cols // 2 if fmt == "mxfp4" else cols
    return dg.MXTensor(FakeTensor((rows, width), torch.uint8, device, Q),
                       FakeTensor((512,), torch.uint8, device, S), cols, fmt)


def test_scales_must_be_where_the_codes_are():
    import torch
    codes = torch.zeros(4, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="one device"):
        dg.MXTensor(codes, torch.zeros(512, dtype=torch.uint8, device="meta"), 64)
    with pytest.raises(ValueError, match="one device"):
        dg.MXTensor(FakeTensor((4, 32), torch.uint8, "cuda:0"),
                    torch.zeros(512, dtype=torch.uint8), 64)


def test_operands_must_be_on_one_device():
    import torch
    q0, q1 = _fake_quantized("cuda:0"), _fake_quantized("cuda:1")
    x = FakeTensor((5, 64), torch.bfloat16, "cuda:0", X)
    dy = FakeTensor((5, 8), torch.bfloat16, "cuda:0", X)
    for f in [lambda: dg.mx_matmul(q0, q1), lambda: dg.mx_linear(x, q1),
              lambda: dg.mx_grad(dy, q1)]:
        with pytest.raises(ValueError, match="one device"):
            f()


@pytest.fixture
def current_device_0():
    """A stand-in for torch that has a current CUDA device, number 0."""
    import types

    import torch
    ext = dg._load_mx()
    names = ("float32", "float16", "bfloat16", "uint8", "empty")
    c = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda index: 0, _cuda_getDevice=lambda: 0)
    ext.setup(types.SimpleNamespace(_C=c, **{n: getattr(torch, n) for n in names}), dg.MXTensor,
              dg.GemmError)
    yield
    ext.setup(torch, dg.MXTensor, dg.GemmError)


def test_operands_must_be_on_the_current_device(current_device_0):
    import torch
    q1 = _fake_quantized("cuda:1")
    x = FakeTensor((5, 64), torch.bfloat16, "cuda:1", X)
    y = FakeTensor((5, 8), torch.bfloat16, "cuda:1", Y)
    for f in [lambda: dg.mx_quantize(x), lambda: dg.mx_dequantize(q1), lambda: dg.mx_matmul(q1, q1),
              lambda: dg.mx_linear(x, q1), lambda: dg.mx_grad(y, q1),
              lambda: dg.mx_dequantize(q1, out=x, stream=16),
              lambda: dg.mx_matmul(q1, q1, out=y, stream=0),
              lambda: dg.mx_linear(x, q1, out=y, stream=16),
              lambda: dg.mx_grad(y, q1, out=x, stream=16)]:
        with pytest.raises(ValueError, match="current CUDA device"):
            f()


@pytest.mark.parametrize("stream,current", [(16, 16), (0, 0), (1, 0), (7 << 20, 7 << 20)])
def test_results_are_allocated_on_the_stream_that_writes_them(monkeypatch, stream, current):
    """With stand-ins for torch's streams and allocation; the calls then fail
    for want of a GPU."""
    import contextlib
    import types

    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    ext, now, seen = dg._load_mx(), [8], []   # torch's current stream is number 8

    @contextlib.contextmanager
    def on(s):
        now.append(s)
        try:
            yield
        finally:
            now.pop()

    def empty(size, dtype=None, device=None):
        seen.append(now[-1])
        return FakeTensor(size if isinstance(size, tuple) else (size,), dtype, device, Y)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=8))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s: s)
    monkeypatch.setattr(torch.cuda, "stream", on)
    c = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda i: now[-1], _cuda_getDevice=lambda: 0)
    names = ("float32", "float16", "bfloat16", "uint8")
    ext.setup(types.SimpleNamespace(_C=c, empty=empty, **{n: getattr(torch, n) for n in names}),
              dg.MXTensor, dg.GemmError)
    try:
        q = _fake_quantized("cuda:0")
        x, dy = (FakeTensor((5, n), torch.bfloat16, "cuda:0", X) for n in (64, 8))
        calls = [lambda s: dg.mx_quantize(x, stream=s), lambda s: dg.mx_dequantize(q, stream=s),
                 lambda s: dg.mx_matmul(q, q, stream=s), lambda s: dg.mx_linear(x, q, stream=s),
                 lambda s: dg.mx_grad(dy, q, stream=s)]
        for s, want in [(stream, current), (8, 8), (None, 8)]:
            for f in calls:
                with pytest.raises(dg.GemmError):
                    f(s)
            assert seen == [want] * len(calls)
            seen.clear()
    finally:
        ext.setup(torch, dg.MXTensor, dg.GemmError)


# ------------------------------------------------------------ the largest sizes

LIMIT = 2 ** 31 - 1024


@pytest.mark.parametrize("K", [LIMIT - 33, LIMIT - 1, LIMIT])
def test_sizes_up_to_the_limit(K):
    assert dg.gemm_mx_code_ld("mxfp4", K) == -(-((K + 1) // 2) // 16) * 16
    assert dg.gemm_mx_code_ld("mxint8", K) == -(-K // 16) * 16
    assert dg.gemm_mx_scale_bytes(1, K) == -(-K // 128) * 512
    assert dg.gemm_mx_scale_bytes(K, 1) == -(-K // 128) * 512


@pytest.mark.parametrize("K", [LIMIT + 1, 2 ** 31 - 16, 2 ** 31 - 1])
def test_sizes_past_the_limit_are_refused(K):
    for fmt in ("mxfp4", "mxint8"):
        assert dg.gemm_mx_code_ld(fmt, K) == -1
        for R, C in [(K, 64), (1, K)]:
            assert _quantize(fmt=fmt, R=R, K=C, ldx=2 ** 31 - 1, ldq=2 ** 31 - 16) == INVALID
            assert dg.gemm_mx_dequantize(fmt, "bf16", R, C, Q, 2 ** 31 - 16, S, Y,
                                         2 ** 31 - 1) == INVALID
    assert dg.gemm_mx_scale_bytes(1, K) == -1 and dg.gemm_mx_scale_bytes(K, 1) == -1
    ld = 2 ** 31 - 16
    for M, N, C in [(K, 8, 64), (4, K, 64), (4, 8, K)]:
        assert dg.gemm_mx4("bf16", M, N, C, 1.0, Q, ld, S, Q2, ld, S2, 0.0, Y, ld) == INVALID
        assert dg.gemm_mx4_linear("bf16", M, N, C, X, ld, Q, ld, S, Y, ld) == INVALID
        assert dg.gemm_mx_grad("mxint8", "bf16", "N", "bf16", M, N, C, 1.0, X, ld, Q, ld, S, 0.0,
                               Y, ld) == INVALID


def test_wrappers_refuse_sizes_past_the_limit(current_device_0):
    import torch
    with pytest.raises(ValueError, match="limit"):
        dg.mx_quantize(FakeTensor((1, 2 ** 31 - 1), torch.bfloat16, "cuda:0", X))
    for shape, cols in [((1, 2 ** 31 - 16), 2 ** 31 - 1), ((2 ** 31 - 1, 16), 16)]:
        with pytest.raises(ValueError, match="limit"):
            dg.MXTensor(FakeTensor(shape, torch.uint8, "cuda:0", Q),
                        FakeTensor((2 ** 40,), torch.uint8, "cuda:0", S), cols)
