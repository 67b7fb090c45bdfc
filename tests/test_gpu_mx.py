"""GPU tests of the microscaled operators against the plain 64-bit
implementation in mx_reference: quantisation and its inverse bit for bit,
the 4-bit product, the linear layer and the products of the backward pass
within a bound derived from FP32 accumulation and one rounding."""
import numpy as np
import pytest
import torch

import mx_reference as ref
from parity import check_device, gpu_lib

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
FMTS = ["mxfp4", "mxint8"]


@pytest.fixture(scope="module")
def dg():
    return gpu_lib()


def _np(t):
    return t.double().cpu().numpy()


def _rand(rng, rows, cols, dtype="f32", spread=3.0):
    """Values over many binades, as a float32 array cast to dtype."""
    x = rng.standard_normal((rows, cols)) * np.exp2(rng.uniform(-spread, spread, (rows, 1)))
    return torch.from_numpy(x.astype(np.float32)).to(TYPES[dtype])


def _dev(t, op="N", pad=0, offset=0):
    """t on the GPU, row-major or stored transposed, rows `pad` elements
    wider than t's and the base `offset` elements into its buffer; the
    padding holds NaN."""
    s = t.t() if op == "T" else t
    rows, cols = s.shape
    buf = torch.full((rows * (cols + pad) + offset + 8,), float("nan"), dtype=t.dtype,
                     device="cuda")
    v = buf[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(s)
    return v.t() if op == "T" else v


def _operand(dg, x, fmt, pad=0):
    """MXTensor of x by the plain implementation, the codes' rows `pad` bytes
    wider, all padding bytes (codes 0xFF past a row's 8-column groups,
    scales 0xFF of rows that do not exist) as a caller may leave them."""
    codes, scales = ref.quantize(x, fmt)
    cb, sb = ref.pack(codes, scales, fmt)
    R, K = x.shape
    wide = np.full((R, cb.shape[1] + pad), 0xFF, dtype=np.uint8)
    width = (K + 1) // 2 if fmt == "mxfp4" else K
    wide[:, :width] = cb[:, :width]
    T = -(-K // 128)
    rows = np.arange(-(-R // 128) * 128).reshape(-1, 4, 32).transpose(0, 2, 1)   # tile, r%32, quad
    gone = np.broadcast_to((rows >= R)[:, None, :, :, None], (rows.shape[0], T, 32, 4, 4))
    sb = np.where(gone.reshape(-1), 0xFF, sb).astype(np.uint8)
    q = dg.MXTensor(torch.from_numpy(wide).cuda(), torch.from_numpy(sb).cuda(), K, fmt)
    return q, ref.values(codes, scales, fmt)


def _check(got, want, total, K, dtype):
    """got within the bound of `want`; NaN exactly where want has it."""
    assert got.dtype == TYPES[dtype] and tuple(got.shape) == want.shape
    got = _np(got)
    nan = np.isnan(want)
    assert (np.isnan(got) == nan).all()
    err = np.abs(np.where(nan, 0, got) - np.where(nan, 0, want))
    lim = ref.bound(np.where(nan, 0, want), np.where(nan, 0, total), K, dtype)
    worst = np.unravel_index(np.argmax(err - lim), err.shape)
    assert (err <= lim).all(), (worst, got[worst], want[worst], lim[worst])


# ------------------------------------------------------------ quantisation

SHAPES = [(1, 1), (1, 32), (3, 33), (1, 4096), (130, 333), (33, 128), (257, 1000), (64, 2080)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("op", ["N", "T"])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_bytes(dg, fmt, dtype, op, shape):
    rng = np.random.default_rng(sum(shape))
    x = _rand(rng, *shape, dtype)
    want_c, want_s = ref.quantize(_np(x), fmt)
    for pad, offset in [(0, 0), (3, 0), (8, 1)]:
        q = dg.mx_quantize(_dev(x, op, pad, offset), fmt)
        check_device(dg)
        c, s = ref.unpack(q.codes.cpu().numpy(), q.scales.cpu().numpy(), shape[1], fmt)
        assert (s == want_s).all()
        same = (c == want_c) if fmt == "mxint8" else \
            (c == want_c) | (((c & 7) == 0) & ((want_c & 7) == 0))   # -0 and 0 stand for 0
        assert same.all()
        if fmt == "mxfp4" and shape[1] % 2:
            assert not (q.codes[:, shape[1] // 2] >> 4).any()
        # The bytes of blocks past a row's last are finite scales.
        full = ref.unpack(q.codes.cpu().numpy(), q.scales.cpu().numpy(),
                          min(-(-shape[1] // 128) * 128, q.codes.shape[1] * 2), "mxfp4")[1]
        assert (full[:, want_s.shape[1]:] != 255).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("op", ["N", "T"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 9), (130, 40), (70, 250), (33, 273), (64, 517)])
def test_quantize_writes_only_its_bytes(dg, fmt, dtype, op, shape):
    """Whole groups of 8 columns of a code row, and the scales of rows that
    exist; what lies between rows belongs to the caller."""
    R, K = shape
    x = _dev(_rand(np.random.default_rng(R), R, K, dtype), op)
    ldq = dg.gemm_mx_code_ld(fmt, K) + 32
    codes = torch.full((R, ldq), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((dg.gemm_mx_scale_bytes(R, K),), 0xA5, dtype=torch.uint8, device="cuda")
    assert dg.gemm_mx_quantize(fmt, dtype, op, R, K, x.data_ptr(), x.stride(1 if op == "T" else 0),
                               codes.data_ptr(), ldq, scales.data_ptr(),
                               torch.cuda.current_stream().cuda_stream) == dg.GEMM_OK
    check_device(dg)
    width = -(-K // 8) * (4 if fmt == "mxfp4" else 8)
    assert (codes[:, width:] == 0xA5).all()
    rows = scales.cpu().numpy().reshape(-(-R // 128), -(-K // 128), 32, 4, 4)
    rows = rows.transpose(0, 3, 2, 1, 4).reshape(-(-R // 128) * 128, -1)
    assert (rows[R:] == 0xA5).all()
    want_c, want_s = ref.quantize(_np(x), fmt)
    c, s = ref.unpack(codes[:, :ldq - 32].cpu().numpy(), scales.cpu().numpy(), K, fmt)
    assert (s == want_s).all()
    np.testing.assert_array_equal(ref.values(c, s, fmt), ref.values(want_c, want_s, fmt))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("op", ["N", "T"])
def test_quantize_special_values(dg, fmt, op):
    x = np.zeros((40, 256), dtype=np.float32)
    x[0, 5] = np.inf
    x[1, 70] = -np.inf
    x[2, 100] = np.nan
    x[3, :] = np.float32(2.0 ** -149)                     # the smallest subnormal
    x[4, :] = np.finfo(np.float32).max
    x[5, :32] = -np.finfo(np.float32).max
    x[6, :] = np.float32(2.0 ** -126)
    x[7, ::2], x[7, 1::2] = 2.0 ** 100, 2.0 ** -100       # far apart in one block
    x[8, :] = -0.0
    grid = np.arange(256) / 32.0                           # every tie of both formats
    x[9, :], x[10, :] = grid, -grid
    x[11, :] = np.linspace(-127.75, 127.75, 256) / 64
    x[12, :32] = np.float32(2.0 ** -127) * 1.5             # subnormal block
    t = torch.from_numpy(x)
    want_c, want_s = ref.quantize(x, fmt)
    q = dg.mx_quantize(_dev(t, op), fmt)
    c, s = ref.unpack(q.codes.cpu().numpy(), q.scales.cpu().numpy(), 256, fmt)
    assert (s == want_s).all()
    want_v = ref.values(want_c, want_s, fmt)
    got_v = ref.values(c, s, fmt)
    np.testing.assert_array_equal(got_v, want_v)
    back = dg.mx_dequantize(q, torch.float32)
    np.testing.assert_array_equal(_np(back), want_v)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", SHAPES)
def test_dequantize_values(dg, fmt, dtype, shape):
    rng = np.random.default_rng(7 + sum(shape))
    q, v = _operand(dg, _np(_rand(rng, *shape)), fmt, pad=16)
    want = torch.from_numpy(v).to(TYPES[dtype])
    buf = torch.full((shape[0], shape[1] + 5), -1.0, dtype=TYPES[dtype], device="cuda")
    for out in [None, buf[:, :shape[1]]]:
        y = dg.mx_dequantize(q, TYPES[dtype], out=out)
        check_device(dg)
        assert torch.equal(y.cpu(), want)
    assert (buf[:, shape[1]:] == -1).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(1, 1), (1, 5), (1, 33), (3, 7), (2, 250), (5, 1001)])
def test_arrays_whose_last_row_ends_with_its_codes(dg, fmt, dtype, shape):
    """The tensor of the codes has no byte past the last row's last code; what
    follows in memory (0xFF here, finite scales' codes) is no part of it."""
    R, K = shape
    x = _np(_rand(np.random.default_rng(K), R, K))
    codes, scales = ref.quantize(x, fmt)
    cb, sb = ref.pack(codes, scales, fmt)
    width = (K + 1) // 2 if fmt == "mxfp4" else K
    pitch = cb.shape[1]
    flat = np.full((R, pitch), 0xFF, dtype=np.uint8)
    flat[:, :width] = cb[:, :width]
    buf = torch.full((R * pitch + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    buf[:R * pitch] = torch.from_numpy(flat.reshape(-1)).cuda()
    tight = buf[:(R - 1) * pitch + width].as_strided((R, width), (pitch, 1))
    q = dg.MXTensor(tight, torch.from_numpy(sb).cuda(), K, fmt)
    want = ref.values(codes, scales, fmt)
    y = dg.mx_dequantize(q, TYPES[dtype])
    check_device(dg)
    assert torch.equal(y.cpu(), torch.from_numpy(want).to(TYPES[dtype]))
    if fmt == "mxfp4" and dtype != "f32":
        a = _rand(np.random.default_rng(1), 3, K, dtype)
        av = ref.values(*ref.quantize(_np(a), fmt), fmt)
        _check(dg.mx_linear(a.cuda(), q), av @ want.T, np.abs(av) @ np.abs(want).T, K, dtype)


def test_dequantize_every_scale(dg):
    """All 256 scales, all codes of both formats; FP16 rounds and overflows."""
    for fmt in FMTS:
        codes = np.tile(np.arange(32) % 16 if fmt == "mxfp4" else np.arange(32) * 8 - 124, (256, 1))
        scales = np.arange(256, dtype=np.uint8)[:, None]
        cb, sb = ref.pack(codes, scales, fmt)
        q = dg.MXTensor(torch.from_numpy(cb).cuda(), torch.from_numpy(sb).cuda(), 32, fmt)
        v = ref.values(codes, scales, fmt)
        for dtype in (torch.float32, torch.bfloat16, torch.float16):
            got = dg.mx_dequantize(q, dtype).cpu()
            want = torch.from_numpy(v).to(torch.float32).to(dtype)
            assert torch.equal(torch.nan_to_num(got, 7.0), torch.nan_to_num(want, 7.0))
            assert (got.isnan() == want.isnan()).all()


# ------------------------------------------------------------ 4-bit product

PRODUCTS = [(1, 1, 1), (1, 128, 32), (2, 3, 31), (128, 128, 256), (33, 77, 130), (129, 130, 333),
            (300, 520, 1024), (1, 1000, 4096), (257, 64, 2000), (1000, 1030, 777),
            (512, 256, 8192), (7, 4097, 160), (640, 2305, 385)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", PRODUCTS)
def test_product(dg, dtype, shape):
    M, N, K = shape
    rng = np.random.default_rng(M + 3 * N + 7 * K)
    a, av = _operand(dg, _np(_rand(rng, M, K)), "mxfp4", pad=16)
    b, bv = _operand(dg, _np(_rand(rng, N, K, spread=1.0)), "mxfp4")
    got = dg.mx_matmul(a, b, dtype=TYPES[dtype])
    check_device(dg)
    _check(got, av @ bv.T, np.abs(av) @ np.abs(bv).T, K, dtype)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(5, 9, 70), (200, 300, 500), (700, 513, 256)])
def test_product_scaled_into_a_padded_view(dg, dtype, shape):
    M, N, K = shape
    rng = np.random.default_rng(5)
    a, av = _operand(dg, _np(_rand(rng, M, K)), "mxfp4")
    b, bv = _operand(dg, _np(_rand(rng, N, K, spread=1.0)), "mxfp4")
    c0 = _rand(rng, M, N, dtype, spread=0.0)
    out = _dev(c0, pad=3, offset=1)
    dg.mx_matmul(a, b, out=out, alpha=0.5, beta=-2.0)
    check_device(dg)
    want = 0.5 * (av @ bv.T) - 2.0 * _np(c0)
    total = 0.5 * (np.abs(av) @ np.abs(bv).T) + 2.0 * np.abs(_np(c0))
    _check(out, want, total, K, dtype)
    whole = out._base if out._base is not None else out
    assert int(whole.isnan().sum()) == whole.numel() - M * N     # padding untouched
    out.fill_(float("nan"))                                      # beta = 0: not read
    dg.mx_matmul(a, b, out=out, alpha=0.5)
    _check(out, 0.5 * (av @ bv.T), total, K, dtype)


def test_products_without_terms(dg):
    e = dg.MXTensor(torch.empty((3, 0), dtype=torch.uint8, device="cuda"),
                    torch.empty(0, dtype=torch.uint8, device="cuda"), 0)
    assert dg.gemm_mx4("f32", 3, 3, 0, 1.0, 0, 0, 0, 0, 0, 0, 0.0, 0, 3) == dg.GEMM_ERR_INVALID_ARG
    out = torch.ones((3, 3), device="cuda")
    dg.mx_matmul(e, e, out=out, beta=2.0)
    assert (out == 2).all()
    dg.mx_matmul(e, e, out=out)
    assert (out == 0).all()
    a, av = _operand(dg, np.ones((3, 40)), "mxfp4")
    out = torch.ones((3, 3), device="cuda")
    dg.mx_matmul(a, a, out=out, alpha=0.0, beta=3.0)
    assert (out == 3).all()
    assert dg.mx_linear(torch.empty((3, 0), dtype=torch.float16, device="cuda"), e).eq(0).all()
    dy = torch.ones((2, 3), dtype=torch.bfloat16, device="cuda")
    out = torch.ones((2, 40), device="cuda")
    dg.mx_grad(dy[:, :0].contiguous(), dg.MXTensor(a.codes[:0], a.scales[:0], 40), out=out)
    assert (out == 0).all()
    assert dg.mx_matmul(a, dg.MXTensor(a.codes[:0], a.scales[:0], 40)).shape == (3, 0)


def test_product_exact_on_integers(dg):
    """Integer values whose sums stay below 2^24: the same bits in FP32."""
    rng = np.random.default_rng(9)
    a = rng.choice([-6, -4, -3, -2, -1, 0, 1, 2, 3, 4, 6], (384, 1100)).astype(np.float64)
    b = rng.choice([-6, -4, -3, -2, -1, 0, 1, 2, 3, 4, 6], (260, 1100)).astype(np.float64)
    a[:, ::32], b[:, ::32] = 4, 6      # every block's scale is 1
    qa, av = _operand(dg, a, "mxfp4")
    qb, bv = _operand(dg, b, "mxfp4")
    assert (av == a).all() and (bv == b).all()
    got = dg.mx_matmul(qa, qb, dtype=torch.float32)
    assert (_np(got) == a @ b.T).all()


def test_product_nan_blocks_stay_in_their_rows(dg):
    rng = np.random.default_rng(11)
    x = rng.standard_normal((200, 300))
    x[17, 40] = np.inf
    w = rng.standard_normal((150, 300))
    w[149, 299] = np.nan
    a, av = _operand(dg, x, "mxfp4")
    b, bv = _operand(dg, w, "mxfp4")
    got = dg.mx_matmul(a, b, dtype=torch.float32)
    total = np.nan_to_num(np.abs(av)) @ np.nan_to_num(np.abs(bv)).T
    _check(got, av @ bv.T, total, 300, "f32")


# ------------------------------------------------------------ linear layer

LINEAR = [(1, 1, 1), (1, 4096, 4096), (1, 1000, 333), (2, 128, 64), (7, 515, 1000),
          (8, 2048, 512), (9, 300, 4096), (16, 256, 8192), (17, 1111, 999), (33, 4096, 4096),
          (64, 640, 2048), (65, 200, 777), (128, 1024, 1024), (300, 1030, 512), (1000, 257, 130)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", LINEAR)
def test_linear(dg, dtype, shape):
    M, N, K = shape
    rng = np.random.default_rng(M + N + K)
    x = _rand(rng, M, K, dtype, spread=2.0)
    w, wv = _operand(dg, _np(_rand(rng, N, K, spread=1.0)), "mxfp4", pad=16)
    xv = ref.values(*ref.quantize(_np(x), "mxfp4"), "mxfp4")
    want, total = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    for pad, offset in [(0, 0), (5, 1)]:
        got = dg.mx_linear(_dev(x, "N", pad, offset), w)
        check_device(dg)
        _check(got, want, total, K, dtype)
    out = torch.full((M, N + 3), -1.0, dtype=TYPES[dtype], device="cuda")
    dg.mx_linear(_dev(x), w, out=out[:, :N])
    _check(out[:, :N], want, total, K, dtype)
    assert (out[:, N:] == -1).all()


# Wide products of short rows: the last size of the few-row kernel and the
# first of the pair kernel, and long rows beside them.
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(56, 2048, 1000), (57, 2048, 1000), (64, 2050, 4096),
                                   (64, 2047, 4096), (64, 2050, 4097), (65, 2047, 300)])
def test_products_around_the_few_row_limit(dg, dtype, shape):
    M, N, K = shape
    rng = np.random.default_rng(M + N + K)
    x = _rand(rng, M, K, dtype, spread=2.0)
    w, wv = _operand(dg, _np(_rand(rng, N, K, spread=1.0)), "mxfp4")
    xv = ref.values(*ref.quantize(_np(x), "mxfp4"), "mxfp4")
    want, total = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    _check(dg.mx_linear(_dev(x), w), want, total, K, dtype)
    _check(dg.mx_matmul(dg.mx_quantize(_dev(x)), w, dtype=TYPES[dtype]), want, total, K, dtype)
    check_device(dg)


# Few rows: the last size that the product's kernel quantises itself and the
# first that is quantised before it, by rows and by length.
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("shape", [(24, 300, 8192), (25, 300, 8192), (33, 129, 7999),
                                   (48, 400, 4096), (49, 400, 4096), (4, 140, 40000),
                                   (5, 140, 40000), (1, 20, 70000)])
def test_linear_few_long_rows(dg, dtype, shape):
    M, N, K = shape
    rng = np.random.default_rng(M + N + K)
    x = _rand(rng, M, K, dtype, spread=2.0)
    w, wv = _operand(dg, _np(_rand(rng, N, K, spread=1.0)), "mxfp4", pad=16)
    xv = ref.values(*ref.quantize(_np(x), "mxfp4"), "mxfp4")
    want, total = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    for pad, offset in [(0, 0), (5, 1)]:
        got = dg.mx_linear(_dev(x, "N", pad, offset), w)
        check_device(dg)
        _check(got, want, total, K, dtype)


@pytest.mark.parametrize("M", [1, 5, 40, 200])
def test_linear_special_rows(dg, M):
    """A token with an infinity or a NaN spoils its own row only; a row of
    zeros gives zeros; scales at both ends of their range."""
    rng = np.random.default_rng(M)
    x = rng.standard_normal((M, 500)).astype(np.float32)
    if M > 1:
        x[1, 499] = np.nan
        x[2:3] = 0
        x[3:4, 64:96] = 2.0 ** -149
        x[4:5] *= 2.0 ** 60
    t = torch.from_numpy(x)
    w, wv = _operand(dg, rng.standard_normal((300, 500)), "mxfp4")
    xv = ref.values(*ref.quantize(x, "mxfp4"), "mxfp4")
    got = dg.mx_linear(t.cuda(), w)
    _check(got, xv @ wv.T, np.nan_to_num(np.abs(xv)) @ np.abs(wv).T, 500, "f32")
    if M == 1:
        t[0, 3] = float("inf")
        assert dg.mx_linear(t.cuda(), w).isnan().all()


# ------------------------------------------------------------ backward products

GRADS = [(1, 1, 1), (1, 40, 7), (16, 128, 64), (33, 77, 130), (256, 128, 64), (129, 300, 257),
         (1000, 1030, 777), (40, 2048, 1000), (640, 512, 96), (300, 264, 4096), (515, 1284, 65)]


def _grad_a(dg, rng, M, K, dtype, op, pad=0):
    a = _rand(rng, M, K, dtype, spread=1.0)
    s = a.t() if op == "T" else a
    rows, cols = s.shape
    buf = torch.full((rows, -(-cols // 8) * 8 + pad), float("nan"), dtype=a.dtype, device="cuda")
    buf[:, :cols] = s.cuda()
    v = buf[:, :cols]
    return a, (v.t() if op == "T" else v)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("op", ["N", "T"])
@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("shape", GRADS)
def test_grad(dg, fmt, dtype, op, out, shape):
    M, N, K = shape
    rng = np.random.default_rng(M + 3 * N + 5 * K)
    a, av = _grad_a(dg, rng, M, K, dtype, op, pad=8)
    b, bv = _operand(dg, _np(_rand(rng, K, N, spread=1.0)), fmt, pad=16)
    bv = _np(torch.from_numpy(bv).to(TYPES[dtype]))
    dc = dtype if out == "same" else "f32"
    got = dg.mx_grad(av, b, dtype=TYPES[dc])
    check_device(dg)
    _check(got, _np(a) @ bv, np.abs(_np(a)) @ np.abs(bv), K, dc)


@pytest.mark.parametrize("fmt,op,dc", [("mxint8", "T", "f32"), ("mxfp4", "N", "bf16"),
                                       ("mxint8", "N", "bf16")])
def test_grad_accumulates_into_a_padded_view(dg, fmt, op, dc):
    M, N, K = 300, 397, 500
    rng = np.random.default_rng(3)
    a, av = _grad_a(dg, rng, M, K, "bf16", op)
    b, bv = _operand(dg, _np(_rand(rng, K, N)), fmt)
    c0 = _rand(rng, M, N, dc, spread=0.0)
    out = _dev(c0, pad=3, offset=1)
    dg.mx_grad(av, b, out=out, alpha=0.25, beta=1.0)
    check_device(dg)
    total = 0.25 * (np.abs(_np(a)) @ np.abs(bv)) + np.abs(_np(c0))
    _check(out, 0.25 * (_np(a) @ bv) + _np(c0), total, K, dc)
    out.fill_(float("nan"))
    dg.mx_grad(av, b, out=out)
    _check(out, _np(a) @ bv, 4 * total, K, dc)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("op", ["N", "T"])
@pytest.mark.parametrize("shape", [(1, 9, 7), (7, 40, 1), (33, 77, 129), (130, 64, 517),
                                   (515, 130, 1003), (300, 256, 20), (1001, 96, 1030)])
def test_grad_of_contiguous_operands(dg, dtype, op, shape):
    """Contiguous A whose rows are no multiple of 16 bytes, as autograd gives
    them, and slices of it that begin at odd addresses: the bits of the
    product with an aligned copy of A."""
    M, N, K = shape
    rng = np.random.default_rng(M + N + K)
    b, bv = _operand(dg, _np(_rand(rng, K, N, spread=1.0)), "mxint8")
    a, av = _grad_a(dg, rng, M, K, dtype, op)
    bv = _np(torch.from_numpy(bv).to(TYPES[dtype]))
    want = dg.mx_grad(av, b, dtype=torch.float32)
    _check(want, _np(a) @ bv, np.abs(_np(a)) @ np.abs(bv), K, "f32")
    rows, cols = (M, K) if op == "N" else (K, M)
    stored = (a if op == "N" else a.t()).contiguous()
    whole = torch.full((rows + 2, cols), float("nan"), dtype=a.dtype, device="cuda")
    for lo in (0, 1, 2):
        if (lo * cols * 2) % 16 and cols % 8 == 0:
            continue
        whole.fill_(float("nan"))
        part = whole[lo:lo + rows]
        part.copy_(stored)
        got = dg.mx_grad(part if op == "N" else part.t(), b, dtype=torch.float32)
        check_device(dg)
        assert torch.equal(got, want)


def test_a_layer_of_odd_width_runs_backward(dg):
    """y of mx_linear, and a gradient of its layout, through autograd."""
    gen = torch.Generator("cuda").manual_seed(2)
    x = torch.randn((70, 130), generator=gen, device="cuda").bfloat16()
    w = dg.mx_quantize(torch.randn((77, 130), generator=gen, device="cuda"))
    y = dg.mx_linear(x, w)
    assert y.is_contiguous() and y.shape == (70, 77)
    y.requires_grad_()
    (y.float() ** 2).sum().backward()
    dy, kept = y.grad, dg.mx_quantize(x, "mxint8")
    wide = torch.zeros((70, 80), dtype=dy.dtype, device="cuda")
    wide[:, :77] = dy
    assert torch.equal(dg.mx_grad(dy, w), dg.mx_grad(wide[:, :77], w))
    assert torch.equal(dg.mx_grad(dy.t(), kept, dtype=torch.float32),
                       dg.mx_grad(wide[:, :77].t(), kept, dtype=torch.float32))


@pytest.mark.parametrize("fmt", FMTS)
def test_grad_every_scale(dg, fmt):
    """Exact in BF16 over the whole range of scales whose values BF16 and
    FP32 hold, one row of B for each scale; NaN blocks; FP16 as rounded."""
    K = 256
    codes = np.tile(np.arange(64) % 16 if fmt == "mxfp4" else np.arange(64) * 4 - 127, (K, 1))
    scales = np.stack([np.arange(K), np.arange(K)[::-1]], axis=1).astype(np.uint8)
    cb, sb = ref.pack(codes, scales, fmt)
    b = dg.MXTensor(torch.from_numpy(cb).cuda(), torch.from_numpy(sb).cuda(), 64, fmt)
    v = ref.values(codes, scales, fmt)
    for dtype in ("bf16", "f16"):
        # One-hot rows pick one row of B each; NaN rows (scale 255) spoil every sum, so
        # they are left out of the contraction here.
        keep = slice(1, 255)
        bk = dg.MXTensor(torch.from_numpy(cb[keep]).cuda(), _scales_of(sb, keep, K).cuda(), 64, fmt)
        a = torch.eye(254, dtype=TYPES[dtype], device="cuda")
        buf = torch.zeros((254, 256), dtype=TYPES[dtype], device="cuda")
        buf[:, :254] = a
        got = dg.mx_grad(buf[:, :254], bk, dtype=torch.float32).cpu()
        want = torch.from_numpy(v[keep]).float().to(TYPES[dtype]).float()
        finite = torch.isfinite(want).all(dim=0)   # (inf * 0 of the other rows is NaN)
        assert torch.equal(got[:, finite], want[:, finite])
        assert got[:, ~finite].isnan().sum() >= (~finite).sum() * 253 if (~finite).any() else True
    eye = torch.eye(256, dtype=torch.bfloat16, device="cuda")
    assert dg.mx_grad(eye, b).isnan().all()


def _scales_of(sb, keep, K):
    """Tiles of the rows `keep` of a K-row, two-block array."""
    r = np.arange(K)
    rows = np.stack([sb[(r // 128) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b]
                     for b in range(2)], axis=1)[keep]
    out = np.zeros(1024, dtype=np.uint8)
    r = np.arange(rows.shape[0])
    for b in range(2):
        out[(r // 128) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b] = rows[:, b]
    return torch.from_numpy(out)


def test_gradients_are_those_of_the_layer(dg):
    """f(x, W) = sum(dY * (x W^T)) with the quantised x and W: mx_grad gives
    its derivatives, by the formula and by differences (f is linear in each,
    so a difference quotient is exact up to rounding)."""
    rng = np.random.default_rng(21)
    T, I, O = 96, 160, 72
    x, w = rng.standard_normal((T, I)), rng.standard_normal((O, I)) / 13
    qx, xv = _operand(dg, x, "mxint8")
    qw, wv = _operand(dg, w, "mxfp4")
    dy = _rand(rng, T, O, "bf16", spread=0.0)
    d = _np(dy)
    dyg = dy.cuda()
    dx = dg.mx_grad(dyg, qw, dtype=torch.float32)
    dw = dg.mx_grad(dyg.t(), qx, dtype=torch.float32)
    _check(dx, d @ wv, np.abs(d) @ np.abs(wv), O, "f32")
    _check(dw, d.T @ xv, np.abs(d).T @ np.abs(xv), T, "f32")

    def f(xx, ww):
        return float((d * (xx @ ww.T)).sum())
    h = 0.5
    for _ in range(4):
        ux, uw = rng.standard_normal((T, I)), rng.standard_normal((O, I))
        num = (f(xv + h * ux, wv) - f(xv - h * ux, wv)) / (2 * h)
        assert abs(num - float((_np(dx) * ux).sum())) <= 1e-5 * np.abs(_np(dx) * ux).sum()
        num = (f(xv, wv + h * uw) - f(xv, wv - h * uw)) / (2 * h)
        assert abs(num - float((_np(dw) * uw).sum())) <= 1e-5 * np.abs(_np(dw) * uw).sum()


# ------------------------------------------------------------ streams, graphs, sizes

def test_other_stream_and_repeated_calls(dg):
    """Calls on a side stream, back to back without waiting, and the same
    bits again on another stream."""
    rng = np.random.default_rng(31)
    x = _rand(rng, 48, 1024, "bf16").cuda()
    w, _ = _operand(dg, rng.standard_normal((512, 1024)), "mxfp4")
    dy = _rand(rng, 48, 512, "bf16", spread=0.0).cuda()
    first = (dg.mx_linear(x, w), dg.mx_grad(dy, w), dg.mx_dequantize(dg.mx_quantize(x, "mxint8")))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(20):
            again = (dg.mx_linear(x, w), dg.mx_grad(dy, w),
                     dg.mx_dequantize(dg.mx_quantize(x, "mxint8")))
    s.synchronize()
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    # Different rows on two streams at once do not share a workspace.
    x2 = (x * 3).contiguous()
    want2 = dg.mx_linear(x2, w)
    torch.cuda.synchronize()
    t = torch.cuda.Stream()
    outs = []
    for _ in range(10):
        with torch.cuda.stream(s):
            a = dg.mx_linear(x, w)
        with torch.cuda.stream(t):
            b = dg.mx_linear(x2, w)
        outs.append((a, b))
    torch.cuda.synchronize()
    for a, b in outs:
        assert torch.equal(a, first[0]) and torch.equal(b, want2)
    check_device(dg)


def test_stream_argument_and_the_allocator(dg):
    """Work on a side stream given as `stream` does not get memory that work of
    the current stream still reads, and its results may be used there."""
    gen = torch.Generator("cuda").manual_seed(9)
    x = torch.randn((64, 4096), generator=gen, device="cuda").bfloat16()
    w = dg.mx_quantize(torch.randn((4096, 4096), generator=gen, device="cuda"))
    want = (dg.mx_quantize(x, "mxint8").codes.clone(), dg.mx_linear(x, w), dg.mx_grad(x, w),
            dg.mx_dequantize(w), dg.mx_matmul(w, w))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        busy = [torch.ones_like(t) for t in want for _ in range(2)]
        torch.cuda._sleep(20_000_000)          # the sums wait here for some milliseconds
        sums = [t.sum(dtype=torch.float64) for t in busy]
        sizes = [t.numel() for t in busy]
        del busy                                # back to the current stream's pool
        s = side.cuda_stream
        q = dg.mx_quantize(x, "mxint8", stream=s)
        got = (q, dg.mx_linear(x, w, stream=s), dg.mx_grad(x, w, stream=s),
               dg.mx_dequantize(w, stream=s), dg.mx_matmul(w, w, stream=s))
        torch.cuda.current_stream().wait_stream(side)
        got = (q.codes,) + got[1:]
        copies = [t.clone() for t in got]
        q.record_stream(torch.cuda.current_stream())
        del q, got
        assert [float(t) for t in sums] == [float(n) for n in sizes]
        for a, b in zip(copies, want):
            assert torch.equal(a, b)
    for s in (0, 1):                            # the default stream by both its names
        assert torch.equal(dg.mx_linear(x, w, stream=s), want[1])
    check_device(dg)


def test_graph_replay(dg):
    """A captured layer step replays on new inputs with the eager bits."""
    rng = np.random.default_rng(41)
    w, _ = _operand(dg, rng.standard_normal((640, 768)), "mxfp4")
    x = _rand(rng, 200, 768, "bf16").cuda()
    dy = _rand(rng, 200, 640, "bf16", spread=0.0).cuda()

    def step():
        kept = dg.mx_quantize(x, "mxint8")
        return dg.mx_linear(x, w), dg.mx_grad(dy, w), dg.mx_grad(dy.t(), kept, dtype=torch.float32)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()          # grows the workspace of this stream
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs = step()
    for seed in (1, 2):
        x.copy_(_rand(np.random.default_rng(seed), 200, 768, "bf16"))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)
    check_device(dg)


def test_arrays_past_32_bit_offsets(dg):
    """More than 2^32 elements: sampled rows of the round trip, and a product
    and a gradient whose operands cross the boundary."""
    R, K = 140000, 32768
    x = torch.empty((R, K), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator("cuda").manual_seed(5)
    for lo in range(0, R, 10000):
        x[lo:lo + 10000] = torch.randn((10000, K), generator=gen, device="cuda")
    rows = [0, 1, 65535, 65536, 131071, 131072, R - 1]
    for fmt in FMTS:
        q = dg.mx_quantize(x, fmt)
        y = dg.mx_dequantize(q)
        xs = _np(x[rows])
        want = ref.values(*ref.quantize(xs, fmt), fmt)
        assert (_np(y[rows]) == want).all()
        if fmt == "mxfp4":
            small, sv = _operand(dg, np.random.default_rng(1).standard_normal((8, K)), "mxfp4")
            got = dg.mx_matmul(q, small, dtype=torch.float32)
            _check(got[rows], want @ sv.T, np.abs(want) @ np.abs(sv).T, K, "f32")
        else:
            # One-hot rows of A pick rows of q: exact.
            a = torch.zeros((len(rows), R), dtype=torch.bfloat16, device="cuda")
            for i, r in enumerate(rows):
                a[i, r] = 1
            got = dg.mx_grad(a, q)
            assert (_np(got) == want).all()
        del q, y
    check_device(dg)


@pytest.mark.parametrize("fmt", FMTS)
def test_one_row_past_32_bit_scale_offsets(dg, fmt):
    """A row of over 2^29 columns, whose scales lie further than 2^31 bytes
    apart: the codes, scales and values of its pieces as short rows."""
    W = 32768
    K = 2 ** 29 + 5 * W + 1037
    gen = torch.Generator("cuda").manual_seed(8)
    x = torch.empty((1, K), dtype=torch.bfloat16, device="cuda")
    for lo in range(0, K, 1 << 27):
        n = min(1 << 27, K - lo)
        x[0, lo:lo + n] = torch.randn(n, generator=gen, device="cuda")
    q = dg.mx_quantize(x, fmt)
    y = dg.mx_dequantize(q)
    check_device(dg)
    body = K // W * W
    per_byte = 2 if fmt == "mxfp4" else 1
    scales = q.scales.view(-1, 512)[:, :4].reshape(-1)      # of row 0, block by block
    for lo, piece in [(0, x[:, :body].view(-1, W)), (body, x[:, body:])]:
        p = dg.mx_quantize(piece, fmt)
        R, C = piece.shape
        n = R * C
        assert torch.equal(y[0, lo:lo + n].view(R, C), dg.mx_dequantize(p))
        width = -(-C // per_byte)
        assert torch.equal(q.codes[0, lo // per_byte:lo // per_byte + R * width],
                           p.codes[:, :width].reshape(-1))
        nb = -(-C // 32)
        s = p.scales.view(-1, -(-nb // 4), 32, 4, 4).permute(0, 3, 2, 1, 4)
        s = s.reshape(s.shape[0] * 128, -1)[:R, :nb].reshape(-1)
        assert torch.equal(scales[lo // 32:lo // 32 + R * nb], s)


# ------------------------------------------------------------ schedules

@pytest.mark.parametrize("shape", [(2100, 2500, 300), (130, 200, 6000), (64, 3000, 2500),
                                   (400, 100, 3000), (4200, 1030, 520)])
def test_product_schedules(dg, shape):
    """Whole tiles with a last round of halves (one of them past M), ranges of
    K summed afterwards, few rows over a cluster; scaled, with an old C."""
    M, N, K = shape
    rng = np.random.default_rng(M)
    a, av = _operand(dg, _np(_rand(rng, M, K, spread=1.0)), "mxfp4")
    b, bv = _operand(dg, _np(_rand(rng, N, K, spread=1.0)), "mxfp4")
    want, total = av @ bv.T, np.abs(av) @ np.abs(bv).T
    for dtype in ("bf16", "f32"):
        _check(dg.mx_matmul(a, b, dtype=TYPES[dtype]), want, total, K, dtype)
        c0 = _rand(rng, M, N, dtype, spread=0.0)
        out = _dev(c0, pad=2)
        dg.mx_matmul(a, b, out=out, alpha=-1.5, beta=0.5)
        check_device(dg)
        _check(out, -1.5 * want + 0.5 * _np(c0), 1.5 * total + 0.5 * np.abs(_np(c0)), K, dtype)


@pytest.mark.parametrize("fmt,op", [("mxint8", "T"), ("mxfp4", "N")])
@pytest.mark.parametrize("shape", [(2100, 2500, 300), (130, 200, 6000), (400, 100, 3000)])
def test_grad_schedules(dg, fmt, op, shape):
    M, N, K = shape
    rng = np.random.default_rng(M + 1)
    a, av = _grad_a(dg, rng, M, K, "bf16", op)
    b, bv = _operand(dg, _np(_rand(rng, K, N, spread=1.0)), fmt)
    want, total = _np(a) @ bv, np.abs(_np(a)) @ np.abs(bv)
    for dtype in ("bf16", "f32"):
        _check(dg.mx_grad(av, b, dtype=TYPES[dtype]), want, total, K, dtype)
        c0 = _rand(rng, M, N, dtype, spread=0.0)
        out = _dev(c0, pad=2)
        dg.mx_grad(av, b, out=out, alpha=-1.5, beta=0.5)
        check_device(dg)
        _check(out, -1.5 * want + 0.5 * _np(c0), 1.5 * total + 0.5 * np.abs(_np(c0)), K, dtype)


def test_long_float32_sums_round_to_nearest(dg):
    """Over 32768 terms the FP32 result keeps the error of sums of 1024 terms
    each, which the tensor cores truncate (a relative error that grows with
    the number of 16-term steps, 64 here), added with rounding: 64 * 2^-23
    of the largest partial sum and 32 * 2^-24 of the running one, over a
    random walk of like terms well under 4e-6 of the result's norm.  Summed
    in one piece it was above 2e-5."""
    rng = np.random.default_rng(77)
    K = 32768
    a = _rand(rng, K, 128, "bf16", spread=0.0)
    b, bv = _operand(dg, rng.standard_normal((K, 96)), "mxint8")
    got = _np(dg.mx_grad(a.cuda().t(), b, dtype=torch.float32))
    want = _np(a).T @ bv
    assert np.linalg.norm(got - want) <= 4e-6 * np.linalg.norm(want)


def test_long_16_bit_sums_keep_their_size(dg):
    """A gradient over 2^19 tokens of like terms, too large for ranges of K:
    what the truncation of each step in tensor memory takes off the results
    stays below 2^-11 * 0.27 = 1.3e-4, a quarter of what FP16 rounds.  (Parts
    of 16384 terms lose 1.0e-4; in one piece it was 3e-3.)"""
    K, M, N = 1 << 19, 8192, 4224
    gen = torch.Generator("cuda").manual_seed(15)
    dy = torch.empty((K, M), dtype=torch.float16, device="cuda")
    x = torch.empty((K, N), dtype=torch.float16, device="cuda")
    step = 1 << 16
    for lo in range(0, K, step):
        dy[lo:lo + step] = torch.rand((step, M), generator=gen, device="cuda") + 0.5
        x[lo:lo + step] = torch.rand((step, N), generator=gen, device="cuda") + 0.5
    kept = dg.mx_quantize(x, "mxint8")
    values = dg.mx_dequantize(kept, torch.float16)
    got = dg.mx_grad(dy.t(), kept, alpha=2.0 ** -19)[:16].double()
    check_device(dg)
    want = torch.zeros((16, N), dtype=torch.float64, device="cuda")
    for lo in range(0, K, step):
        want += dy[lo:lo + step, :16].double().t() @ values[lo:lo + step].double()
    want *= 2.0 ** -19
    assert abs(float(((got - want) / want).mean())) <= 1.3e-4


@pytest.mark.parametrize("M,N,linear", [(2048, 2048, False), (8, 19600, False), (2, 19600, True),
                                        (40, 260, False), (1, 260, True)])
def test_long_float32_products_of_far_scales(dg, M, N, linear):
    """Blocks whose scales lie up to 24 binades apart, so that no sum fits the
    24 bits of FP32, over 32768 terms.  The tensor cores drop up to 2^-23 of
    the running sum at each 64-deep step, on average half of that; a result
    keeps at most 64 such steps (the sum of 4096 terms) and adds its at most
    eight parts with 2^-24 each: 64 * 2^-24 + 8 * 2^-24 = 4.3e-6 of the
    largest partial sums, which are below the result's norm in a random walk.
    (In one piece, as with the first two shapes, it was 1e-5.)"""
    K = 32768
    gen = torch.Generator("cuda").manual_seed(12)

    def rand(rows):
        x = torch.randn((rows, K), generator=gen, device="cuda")
        e = torch.randint(-12, 13, (rows, K // 32), generator=gen, device="cuda")
        return (x.view(rows, -1, 32) * torch.exp2(e.float()).unsqueeze(-1)).view(rows, K)
    x = rand(M)
    b = dg.mx_quantize(rand(N))
    a = dg.mx_quantize(x)
    got = dg.mx_linear(x, b) if linear else dg.mx_matmul(a, b, dtype=torch.float32)
    check_device(dg)
    rows, cols = slice(0, 64), slice(0, N, max(N // 512, 1))
    av = dg.mx_dequantize(a, torch.float32)[rows].double()
    want = av @ dg.mx_dequantize(b, torch.float32)[cols].double().t()
    assert (got[rows, cols].double() - want).norm() <= 4.3e-6 * want.norm()


def test_refusals_of_the_wrappers(dg):
    x = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    q4, q8 = dg.mx_quantize(x), dg.mx_quantize(x, "mxint8")
    wide = torch.zeros((8, 8, 4), dtype=torch.bfloat16, device="cuda")
    bad = [
        lambda: dg.mx_quantize(x, "mxfp6"), lambda: dg.mx_quantize(x.cpu()),
        lambda: dg.mx_quantize(x.double()), lambda: dg.mx_quantize(wide),
        lambda: dg.mx_quantize(wide[:, :, 1]),                      # no unit stride
        lambda: dg.mx_dequantize(x), lambda: dg.mx_dequantize(q4, torch.int8),
        lambda: dg.mx_dequantize(q4, out=torch.zeros((8, 63), device="cuda")),
        lambda: dg.mx_dequantize(q4, torch.float16, out=torch.zeros((8, 64), device="cuda")),
        lambda: dg.mx_matmul(q4, q8), lambda: dg.mx_matmul(q4, q4, beta=1.0),
        lambda: dg.mx_matmul(q4, dg.mx_quantize(x[:, :32])),
        lambda: dg.mx_matmul(q4, q4, out=torch.zeros((8, 8))),
        lambda: dg.mx_linear(x, q8), lambda: dg.mx_linear(x[:, :32], q4),
        lambda: dg.mx_linear(x.t(), dg.mx_quantize(torch.zeros((5, 8), device="cuda"))),
        lambda: dg.mx_linear(x, q4, out=torch.zeros((8, 8), device="cuda")),
        lambda: dg.mx_grad(x.float(), q4), lambda: dg.mx_grad(x, q4),
        lambda: dg.mx_grad(x[:, :8], q4, dtype=torch.float16),
        lambda: dg.mx_grad(x[:, :8], q4, beta=1.0), lambda: dg.mx_grad(wide[:, :, 1], q4),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    shifted = torch.zeros(8 * 64 + 8, dtype=torch.bfloat16, device="cuda")[1:513].view(8, 64)
    for f, status in [(lambda: dg.mx_grad(shifted[:, :8], q4), dg.GEMM_ERR_MISALIGNED),
                      (lambda: dg.mx_grad(torch.zeros((8, 17), dtype=torch.bfloat16,
                                                      device="cuda")[:, :8], q4),
                       dg.GEMM_ERR_MISALIGNED),
                      (lambda: dg.mx_quantize(x[:1].expand(8, 64)), dg.GEMM_ERR_INVALID_ARG)]:
        with pytest.raises(dg.GemmError) as e:
            f()
        assert e.value.status == status
    check_device(dg)
