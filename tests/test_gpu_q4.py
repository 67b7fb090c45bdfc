"""GPU tests of the products with 4-bit weights and group scales against plain
64-bit products with the weights' values."""
import pytest
import torch

import mx_reference as ref
from parity import check_device, gpu_lib

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
NAN = float("nan")


@pytest.fixture(scope="module")
def dg():
    return gpu_lib()


def _offsets(sizes, first=0):
    ends = [first]
    for n in sizes:
        ends.append(ends[-1] + n)
    return torch.tensor(ends, dtype=torch.int32, device="cuda")


def _x(gen, rows, K, dtype, pad=8):
    """Normal values in rows `pad` elements wider than a multiple of 8; the padding is
    NaN."""
    buf = torch.full((rows, -(-K // 8) * 8 + pad), NAN, dtype=TYPES[dtype], device="cuda")
    v = buf[:, :K]
    v.copy_(torch.randn((rows, K), generator=gen, device="cuda"))
    return v


def _weights(dg, gen, lead, K, dtype, group, zeros, pad=0):
    """A Q4Tensor and its values in 64 bits.  Bytes past a row's last code, and the
    high half of an odd row's last one, are random as all others; the high bits of
    the zeros are set."""
    pitch = -(-((K + 1) // 2) // 16) * 16 + pad
    codes = torch.randint(0, 256, (*lead, pitch), generator=gen, device="cuda", dtype=torch.uint8)
    n = -(-K // group)
    scales = (torch.randn((*lead, n), generator=gen, device="cuda") * 0.1).to(TYPES[dtype])
    z = None
    if zeros:
        z = torch.randint(0, 16, (*lead, n), generator=gen, device="cuda", dtype=torch.uint8)
    k = torch.arange(K, device="cuda")
    q = (codes[..., k // 2].int() >> (4 * (k % 2)).int()) & 15
    zz = 8 if z is None else z[..., k // group].int()
    values = scales[..., k // group].double() * (q - zz).double()
    if z is not None:
        z = z | 0xF0
    return dg.Q4Tensor(codes, scales, z, cols=K, group=group), values


def _check(got, x, values, K, dtype, rounded=True):
    """got within the bound of x . values^T.  rounded: the weights may have been
    rounded to dtype (half a unit each), as they are for more than FEW rows.  A group's
    sum is multiplied by its scale and added to a running sum: two more roundings of
    FP32 for every 32 terms."""
    p, total = x.double() @ values.t(), x.double().abs() @ values.abs().t()
    lim = torch.from_numpy(ref.bound(p.cpu().numpy(), total.cpu().numpy(), 2 * K + 512, dtype))
    if rounded:
        lim = lim + ref.UNIT[dtype] * total.cpu() * (1 + ref.UNIT[dtype])
        if dtype == "f16":     # and half the smallest subnormal of each
            lim = lim + 2.0 ** -25 * x.double().abs().sum(1, keepdim=True).cpu()
    err = (got.double().cpu() - p.cpu()).abs()
    bad = ~(err <= lim)
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError((int(bad.sum()), at, float(got[at]), float(p[at]), float(lim[at])))


DENSE = [(1, 1, 1, 32), (1, 64, 512, 128), (3, 65, 33, 32), (8, 200, 1000, 64), (9, 64, 544, 96),
         (16, 130, 4096, 128), (17, 129, 777, 32), (25, 64, 2050, 64), (33, 100, 640, 128),
         (48, 64, 512, 64), (64, 300, 1024, 1024), (65, 100, 333, 64), (100, 64, 96, 4096),
         (128, 257, 1500, 128), (300, 300, 500, 32), (513, 64, 1031, 128)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("shape", DENSE, ids=str)
def test_dense(dg, dtype, zeros, shape):
    rows, N, K, group = shape
    gen = torch.Generator("cuda").manual_seed(rows * 7 + N + K)
    x = _x(gen, rows, K, dtype)
    w, values = _weights(dg, gen, (N,), K, dtype, group, zeros, pad=16)
    wide = torch.full((rows + 2, N + 5), 7.0, dtype=TYPES[dtype], device="cuda")
    y = wide[1:rows + 1, 2:2 + N]
    assert dg.q4_linear(x, w, out=y) is y
    check_device(dg)
    inside = torch.zeros_like(wide, dtype=torch.bool)
    inside[1:rows + 1, 2:2 + N] = True
    assert (wide[~inside] == 7.0).all()
    _check(y, x, values, K, dtype, rows > 8)
    assert torch.equal(dg.q4_linear(x, w), y)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows", [7, 16, 40])
def test_long_rows(dg, dtype, group, rows):
    """Rings that go round several times, on all SMs at once, over and over: every
    pass has the same bits, within the bound."""
    gen = torch.Generator("cuda").manual_seed(rows + group)
    x = _x(gen, rows, 8192, dtype)
    w, values = _weights(dg, gen, (8192,), 8192, dtype, group, True)
    y = dg.q4_linear(x, w)
    _check(y, x, values, 8192, dtype, rows > 8)
    for _ in range(5):
        assert torch.equal(dg.q4_linear(x, w), y)
    check_device(dg)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,N,K", [
    (5, 6400, 1600), (3, 3800, 2600), (7, 2700, 3600), (8, 200, 4096), (1, 2400, 3100),
    (16, 5000, 2000), (11, 3300, 2300), (40, 5120, 2100), (20, 3200, 1541), (100, 2500, 1800),
    (65, 2000, 1900), (33, 2048, 4096), (17, 200, 8000)])
def test_shares_of_long_rows(dg, dtype, rows, N, K):
    """Rows of W shared by clusters of every number of CTAs that occurs."""
    gen = torch.Generator("cuda").manual_seed(rows + N + K)
    x = _x(gen, rows, K, dtype)
    w, values = _weights(dg, gen, (N,), K, dtype, 64, True)
    y = dg.q4_linear(x, w)
    check_device(dg)
    _check(y, x, values, K, dtype)
    assert torch.equal(dg.q4_linear(x, w), y)


EXPERTS = [([1], 64, 64, 32), ([0, 1, 0, 2], 130, 520, 64), ([0, 0], 64, 64, 32),
           ([3, 0, 9, 1, 40], 65, 777, 32), ([1] * 33, 64, 300, 128), ([70, 0, 1, 200], 100, 512, 64),
           ([300, 0, 500, 7], 129, 777, 96), ([0, 1500], 64, 96, 32),
           ([5000, 0, 2500, 700], 100, 333, 64)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("case", EXPERTS, ids=lambda c: f"{len(c[0])}x{sum(c[0])}-{c[1]}-{c[2]}")
def test_experts(dg, dtype, zeros, case):
    """Rows outside the groups are NaN and the experts without rows have NaN scales:
    none of it shows, and those rows of the result keep what they held."""
    sizes, N, K, group = case
    gen = torch.Generator("cuda").manual_seed(sum(sizes) + N + K)
    first, rows = 2, sum(sizes) + 2 + 9
    x = _x(gen, rows, K, dtype)
    x[:first] = NAN
    x[first + sum(sizes):] = NAN
    w, values = _weights(dg, gen, (len(sizes), N), K, dtype, group, zeros)
    for g, n in enumerate(sizes):
        if n == 0:
            w.scales[g] = NAN
    y = torch.full((rows, N), 7.0, dtype=TYPES[dtype], device="cuda")
    dg.q4_linear(x, w, offsets=_offsets(sizes, first), out=y)
    check_device(dg)
    assert (y[:first] == 7.0).all() and (y[first + sum(sizes):] == 7.0).all()
    lo = first
    for g, n in enumerate(sizes):
        if n:
            _check(y[lo:lo + n], x[lo:lo + n], values[g], K, dtype, True)
        lo += n


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("K", [64, 256, 4096])
@pytest.mark.parametrize("sizes", [[2, 0, 3, 1], [30, 0, 9, 61], [3000, 0, 2500, 2900]],
                         ids=lambda s: str(sum(s)))
def test_experts_with_the_largest_group(dg, zeros, K, sizes):
    """A scale for each row, by a group that K is far below: K + group - 1 is past what an
    int holds.  Rows for each of the kernels."""
    gen = torch.Generator("cuda").manual_seed(sum(sizes) + K)
    x = _x(gen, sum(sizes), K, "bf16")
    w, values = _weights(dg, gen, (len(sizes), 70), K, "bf16", 2 ** 31 - 32, zeros)
    y = dg.q4_linear(x, w, offsets=_offsets(sizes))
    check_device(dg)
    lo = 0
    for g, n in enumerate(sizes):
        if n:
            _check(y[lo:lo + n], x[lo:lo + n], values[g], K, "bf16", sum(sizes) > 8)
        lo += n


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group,K", [(32, 1600), (64, 130), (128, 2000)])
@pytest.mark.parametrize("experts,N", [(64, 1100), (1024, 200)])
def test_more_tiles_of_experts_than_run_at_once(dg, dtype, group, K, experts, N):
    """Experts of 0 to 3 rows and one of 70, in several rounds."""
    gen = torch.Generator("cuda").manual_seed(experts + K)
    sizes = torch.randint(0, 4, (experts,), generator=gen, device="cuda").tolist()
    sizes[5] = 70
    x = _x(gen, sum(sizes), K, dtype)
    w, values = _weights(dg, gen, (experts, N), K, dtype, group, True)
    y = dg.q4_linear(x, w, offsets=_offsets(sizes))
    for _ in range(3):
        assert torch.equal(dg.q4_linear(x, w, offsets=_offsets(sizes)), y)
    check_device(dg)
    ends = torch.tensor([0] + sizes).cumsum(0).tolist()
    for g in [0, 1, 2, 3, 4, 5, 6, experts // 2, experts - 3, experts - 2, experts - 1]:
        lo, hi = ends[g], ends[g + 1]
        if hi > lo:
            _check(y[lo:hi], x[lo:hi], values[g], K, dtype, True)
    every = torch.arange(experts, device="cuda").repeat_interleave(
        torch.tensor(sizes, device="cuda"))
    want = torch.stack([values[g] @ r for g, r in zip(every.tolist(), x.double())])
    assert float((y.double() - want).norm() / want.norm()) <= 2 * ref.UNIT[dtype]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,N,K,group", [
    (12, 70000, 256, 64), (16, 40001, 424, 32), (30, 40000, 200, 128), (25, 50000, 700, 32),
    (60, 40000, 130, 32), (40, 30000, 1100, 128), (100, 33000, 40, 32), (2000, 4100, 100, 32),
    (1000, 8200, 256, 128), (300, 16400, 520, 64), (1500, 3000, 1290, 128)])
def test_more_tiles_than_run_at_once(dg, dtype, rows, N, K, group):
    """Several units for each CTA, from two k-tiles each on: the same bits every time."""
    gen = torch.Generator("cuda").manual_seed(rows + N + K)
    x = _x(gen, rows, K, dtype)
    w, values = _weights(dg, gen, (N,), K, dtype, group, True)
    y = dg.q4_linear(x, w)
    for _ in range(3):
        assert torch.equal(dg.q4_linear(x, w), y)
    check_device(dg)
    for at in (slice(0, 300), slice(N // 2, N // 2 + 300), slice(N - 300, N)):
        _check(y[:, at], x, values[at], K, dtype)
    want = x.double() @ values.t()
    # (Each weight and each result is off by half a unit at most.)
    assert float((y.double() - want).norm() / want.norm()) <= 2 * ref.UNIT[dtype]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("group,K", [(32, 96), (64, 300), (128, 1000)])
def test_more_tiles_of_experts_than_run_at_once_on_tcgen05(dg, dtype, group, K):
    """Experts of 0 to 60 rows, several units for each CTA, and rows of none around them."""
    gen = torch.Generator("cuda").manual_seed(K)
    sizes = torch.randint(0, 61, (70,), generator=gen, device="cuda").tolist()
    sizes[3] = 0
    sizes[69] = 0
    x = _x(gen, sum(sizes) + 11, K, dtype)
    w, values = _weights(dg, gen, (70, 1300), K, dtype, group, True)
    y = torch.full((sum(sizes) + 11, 1300), 7.0, dtype=TYPES[dtype], device="cuda")
    off = _offsets(sizes, 4)
    for i in range(3):
        got = dg.q4_linear(x, w, offsets=off, out=y.clone())
        assert i == 0 or torch.equal(got, last)
        last = got
    check_device(dg)
    assert (got[:4] == 7.0).all() and (got[4 + sum(sizes):] == 7.0).all()
    lo = 4
    for g, n in enumerate(sizes):
        if n and g % 6 == 0:
            _check(got[lo:lo + n], x[lo:lo + n], values[g], K, dtype)
        lo += n


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows,N,K,group", [(2050, 130, 257, 32), (4100, 65, 300, 128)])
def test_many_rows(dg, dtype, zeros, rows, N, K, group):
    gen = torch.Generator("cuda").manual_seed(rows + N + K)
    x = _x(gen, rows, K, dtype)
    w, values = _weights(dg, gen, (N,), K, dtype, group, zeros, pad=16)
    _check(dg.q4_linear(x, w), x, values, K, dtype)
    check_device(dg)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 7, 12, 40, 64, 200, 2100])
def test_exact_on_integers(dg, dtype, rows):
    """Integer activations and power-of-two scales: FP32 holds every sum exactly, so
    the result is the exact one, rounded once."""
    gen = torch.Generator("cuda").manual_seed(rows)
    N, K, group = 200, 1056, 32
    x = torch.randint(-3, 4, (rows, K), generator=gen, device="cuda").to(TYPES[dtype])
    w, _ = _weights(dg, gen, (N,), K, dtype, group, True)
    w.scales.copy_(2.0 ** torch.randint(-3, 2, w.scales.shape, generator=gen, device="cuda"))
    k = torch.arange(K, device="cuda")
    q = (w.codes[:, k // 2].int() >> (4 * (k % 2)).int()) & 15
    values = w.scales[:, k // group].double() * (q - (w.zeros[:, k // group] & 15).int()).double()
    assert torch.equal(dg.q4_linear(x, w), (x.double() @ values.t()).to(TYPES[dtype]))
    check_device(dg)


@pytest.mark.parametrize("rows", [2, 40, 200, 2100])
def test_special_values_stay_in_their_row_and_column(dg, rows):
    """An infinity or a NaN in a row of x, and a NaN scale of a row of W."""
    gen = torch.Generator("cuda").manual_seed(4)
    x = _x(gen, rows, 512, "bf16")
    w, values = _weights(dg, gen, (130,), 512, "bf16", 64, True)
    w.scales[77, 3] = NAN
    x[1, 100] = NAN
    y = dg.q4_linear(x, w)
    assert y[1].isnan().all() and y[:, 77].isnan().all()
    keep_r = torch.tensor([r for r in range(rows) if r != 1], device="cuda")
    keep_c = torch.tensor([c for c in range(130) if c != 77], device="cuda")
    _check(y[keep_r][:, keep_c], x[keep_r], values[keep_c], 512, "bf16", rows > 8)
    check_device(dg)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,K", [(1, 100), (20, 1), (20, 100), (40, 1031), (100, 157), (800, 100)])
def test_scales_whose_codes_past_the_end_would_overflow(dg, dtype, rows, K):
    """Codes 7 to 9 of scales of 9000: the weights are finite, 8 times the scale is not in
    FP16.  Nothing past a row's last code counts, whatever it stands for."""
    gen = torch.Generator("cuda").manual_seed(rows + K)
    x = (_x(gen, rows, K, "bf16") * 0.01).to(TYPES[dtype])
    buf = torch.full((rows, -(-K // 8) * 8 + 8), NAN, dtype=TYPES[dtype], device="cuda")
    buf[:, :K] = x
    n = -(-K // 128)
    codes = torch.randint(0, 256, (130, -(-K // 32) * 16), generator=gen, device="cuda",
                          dtype=torch.uint8)
    k = torch.arange(K, device="cuda")
    q = torch.randint(7, 10, (130, K), generator=gen, device="cuda")
    for half in (0, 1):
        at = k[k % 2 == half]
        keep = 0xF0 if half == 0 else 0x0F
        codes[:, at // 2] = (codes[:, at // 2] & keep) | (q[:, at] << (4 * half)).to(torch.uint8)
    scales = torch.full((130, n), 9000.0, device="cuda").to(TYPES[dtype])
    w = dg.Q4Tensor(codes, scales, cols=K, group=128)
    values = scales[:, k // 128].double() * (q - 8).double()
    _check(dg.q4_linear(buf[:, :K], w), buf[:, :K], values, K, dtype, rows > 8)
    check_device(dg)


@pytest.mark.parametrize("rows", [1, 5, 70, 300, 2100])
def test_contiguous_x_of_any_width(dg, rows):
    gen = torch.Generator("cuda").manual_seed(5)
    x = torch.randn((rows, 333), generator=gen, device="cuda").half()
    w, values = _weights(dg, gen, (96,), 333, "f16", 64, True)
    _check(dg.q4_linear(x, w), x, values, 333, "f16", rows > 8)
    buf = torch.randn(rows * 512 + 1, generator=gen, device="cuda").half()
    x = buf[1:].view(rows, 512)                       # packed, not 16-byte aligned
    w, values = _weights(dg, gen, (96,), 512, "f16", 64, False)
    _check(dg.q4_linear(x, w), x, values, 512, "f16", rows > 8)
    check_device(dg)


def test_empty_calls(dg):
    gen = torch.Generator("cuda").manual_seed(6)
    w, _ = _weights(dg, gen, (32,), 64, "bf16", 32, True)
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    assert dg.q4_linear(x[:0], w).shape == (0, 32)
    none = dg.Q4Tensor(torch.zeros((32, 16), dtype=torch.uint8, device="cuda"),
                       torch.zeros((32, 0), dtype=torch.bfloat16, device="cuda"), cols=0)
    assert (dg.q4_linear(x[:, :0], none) == 0).all()
    none = dg.Q4Tensor(torch.zeros((2, 32, 16), dtype=torch.uint8, device="cuda"),
                       torch.zeros((2, 32, 0), dtype=torch.bfloat16, device="cuda"), cols=0)
    y = torch.full((4, 32), 7.0, dtype=torch.bfloat16, device="cuda")
    dg.q4_linear(x[:, :0], none, offsets=_offsets([1, 2]), out=y)
    assert (y[:3] == 0).all() and (y[3] == 7).all()
    check_device(dg)


def test_weights_without_rows(dg):
    """Experts of no outputs, and of one, whose codes' rows are the experts' distance."""
    gen = torch.Generator("cuda").manual_seed(16)
    x = _x(gen, 5, 64, "bf16")
    none = dg.Q4Tensor(torch.zeros((3, 0, 32), dtype=torch.uint8, device="cuda"),
                       torch.zeros((3, 0, 1), dtype=torch.bfloat16, device="cuda"))
    assert dg.q4_linear(x, none, offsets=_offsets([1, 2, 2])).shape == (5, 0)
    w, values = _weights(dg, gen, (3, 1), 64, "bf16", 32, True, pad=16)
    y = dg.q4_linear(x, w, offsets=_offsets([1, 2, 2]))
    for g, (lo, hi) in enumerate(((0, 1), (1, 3), (3, 5))):
        _check(y[lo:hi], x[lo:hi], values[g], 64, "bf16")
    check_device(dg)


@pytest.mark.parametrize("rows", [10, 700, 7000])
@pytest.mark.parametrize("raw,meant", [([0, 5, 3, 9], [0, 5, 5, 9]), ([-4, 2, 6, 9], [0, 2, 6, 9]),
                                       ([0, 5000, 6, 9], [0, -1, -1, -1])])
def test_bad_offsets_stay_inside_and_are_reported(dg, rows, raw, meant):
    gen = torch.Generator("cuda").manual_seed(9)
    x = _x(gen, rows, 64, "bf16")
    w, _ = _weights(dg, gen, (3, 64), 64, "bf16", 32, True)
    # (5000 becomes the number of rows, or stays where there are more: then it is in range.)
    meant = [min(rows, 5000) if v < 0 else v for v in meant]
    outs = []
    for offsets in (raw, meant):
        y = torch.full((rows, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        dg.q4_linear(x, w, out=y, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
        st, bits = dg.gemm_device_check(torch.cuda.current_stream().cuda_stream)
        assert (st, bits) == ((dg.GEMM_ERR_DEVICE_TIMEOUT, 1 << 9) if offsets is raw
                              else (dg.GEMM_OK, 0))
        outs.append(y)
    assert torch.equal(*outs)


def test_graph_replay_with_other_groups(dg):
    gen = torch.Generator("cuda").manual_seed(12)
    cases = []
    for rows, experts in ((30, 6), (900, 3), (6400, 3)):
        w, _ = _weights(dg, gen, (experts, 200), 544, "bf16", 32, True)
        cases.append((_x(gen, rows, 544, "bf16"), w, _offsets([rows // experts] * experts)))
    dense = [(_x(gen, rows, 544, "bf16"), _weights(dg, gen, (200,), 544, "bf16", 32, True)[0], None)
             for rows in (3, 300, 2100)]

    def step():
        return [dg.q4_linear(x, w, offsets=o) for x, w, o in cases + dense]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs = step()
    for share in ((1.0, 0.0, 0.0), (0.1, 0.3, 0.6)):
        for x, w, o in cases:
            sizes = [int(f * x.shape[0]) for f in share] + [0] * (w.experts - 3)
            sizes[-1] += x.shape[0] - sum(sizes)
            o.copy_(_offsets(sizes))
            x.normal_(generator=gen)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b)
    check_device(dg)


def test_stream_argument_and_the_allocator(dg):
    gen = torch.Generator("cuda").manual_seed(13)
    xs = [_x(gen, rows, 1024, "bf16") for rows in (4, 400, 4100)]
    w, _ = _weights(dg, gen, (4096,), 1024, "bf16", 128, True)
    want = [dg.q4_linear(x, w) for x in xs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        busy = [torch.ones_like(t) for t in want for _ in range(2)]
        torch.cuda._sleep(20_000_000)
        sums, sizes = [t.sum(dtype=torch.float64) for t in busy], [t.numel() for t in busy]
        del busy
        got = [dg.q4_linear(x, w, stream=side.cuda_stream) for x in xs]
        torch.cuda.current_stream().wait_stream(side)
        copies = [t.clone() for t in got]
        del got
        assert [float(t) for t in sums] == [float(n) for n in sizes]
        for a, b in zip(copies, want):
            assert torch.equal(a, b)
    check_device(dg)


def test_two_streams_at_once(dg):
    """Products with 4-bit weights of every kernel on one stream, others that use tensor
    memory on another."""
    gen = torch.Generator("cuda").manual_seed(17)
    w, _ = _weights(dg, gen, (1024,), 4096, "bf16", 128, True)
    e, _ = _weights(dg, gen, (4, 512), 1024, "bf16", 32, True)
    m = dg.mx_quantize(torch.randn((1024, 4096), generator=gen, device="cuda").bfloat16())
    g = torch.randn((4, 1024, 512), generator=gen, device="cuda").bfloat16()
    xs = [_x(gen, rows, 4096, "bf16") for rows in (5, 16, 33, 100, 900, 4100)]
    r = _x(gen, 70, 1024, "bf16")
    packed = torch.randn((33, 4095), generator=gen, device="cuda").bfloat16()
    wp, _ = _weights(dg, gen, (200,), 4095, "bf16", 128, True)
    off = _offsets([30, 0, 15, 25])

    def one():
        return [dg.q4_linear(x, w) for x in xs] + [dg.q4_linear(r, e, offsets=off),
                                                   dg.q4_linear(packed, wp)]

    def two():
        return ([dg.mx_linear(x.contiguous(), m) for x in xs[:4]] + [dg.grouped_matmul(r, g, off)]
                + [dg.q4_linear(x, w) for x in xs])
    want = one(), two()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s, f in zip(streams, (one, two)):
            with torch.cuda.stream(s):
                got.append(f())
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        for a, b in zip(outs, want[i % 2]):
            assert torch.equal(a, b)
    check_device(dg)


def test_arrays_past_32_bit_offsets(dg):
    """Codes past 2^32 bytes, more weights than the workspace holds at a time."""
    gen = torch.Generator("cuda").manual_seed(14)
    E, N, K, group = 20, 16384, 30000, 64
    codes = torch.zeros((E, N, 15008), dtype=torch.uint8, device="cuda")      # 4.9e9
    codes[E - 1] = torch.randint(0, 256, (N, 15008), generator=gen, device="cuda",
                                 dtype=torch.uint8)
    scales = torch.ones((E, N, -(-K // group)), dtype=torch.bfloat16, device="cuda")
    zeros = torch.randint(0, 16, scales.shape, generator=gen, device="cuda", dtype=torch.uint8)
    w = dg.Q4Tensor(codes, scales, zeros, cols=K, group=group)
    k = torch.arange(K, device="cuda")
    at = torch.arange(0, N, 331, device="cuda")
    for rows in (12, 1500):
        sizes = [1] + [0] * (E - 3) + [2, rows - 3]
        x = _x(gen, rows, K, "bf16")
        y = dg.q4_linear(x, w, offsets=_offsets(sizes))
        check_device(dg)
        lo = 0
        for g, n in enumerate(sizes):
            if n:
                c = codes[g][at]
                q = (c[:, k // 2].int() >> (4 * (k % 2)).int()) & 15
                values = (q - zeros[g][at][:, k // group].int()).double()
                _check(y[lo:lo + n][:, at], x[lo:lo + n], values, K, "bf16", True)
            lo += n


def test_one_matrix_larger_than_the_workspace(dg):
    gen = torch.Generator("cuda").manual_seed(15)
    N, K = 9000, 16384                                       # 295 MB in 16 bits
    w, values = _weights(dg, gen, (N,), K, "f16", 128, True)
    x = _x(gen, 300, K, "f16")
    y = dg.q4_linear(x, w)
    check_device(dg)
    _check(y, x, values, K, "f16", True)


def test_refusals_of_the_wrappers(dg):
    def u8(*shape):
        return torch.zeros(shape, dtype=torch.uint8, device="cuda")

    def s(*shape):
        return torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    q, e = dg.Q4Tensor(u8(8, 32), s(8, 2), group=32), dg.Q4Tensor(u8(2, 8, 32), s(2, 8, 2), group=32)
    assert q.shape == (8, 64) and e.shape == (2, 8, 64) and q.device == u8(1).device
    x, off = s(4, 64), _offsets([1, 1])
    bad = [
        lambda: dg.Q4Tensor(u8(8), s(1)), lambda: dg.Q4Tensor(s(8, 32), s(8, 1)),
        lambda: dg.Q4Tensor(u8(8, 32).cpu(), s(8, 1).cpu()), lambda: dg.Q4Tensor(u8(8, 32), s(8, 2)),
        lambda: dg.Q4Tensor(u8(8, 32), s(8, 1).float()), lambda: dg.Q4Tensor(u8(8, 32), s(8, 1).cpu()),
        lambda: dg.Q4Tensor(u8(8, 32), s(8, 2), group=48), lambda: dg.Q4Tensor(u8(8, 32), s(8, 2), group=0),
        lambda: dg.Q4Tensor(u8(8, 32), s(8, 1), cols=65), lambda: dg.Q4Tensor(u8(8, 32), s(8, 0), cols=-1),
        lambda: dg.Q4Tensor(u8(8, 24), s(8, 1)), lambda: dg.Q4Tensor(u8(8, 64)[:, ::2], s(8, 1)),
        lambda: dg.Q4Tensor(u8(8, 33)[:, 1:], s(8, 1)), lambda: dg.Q4Tensor(u8(1, 32).expand(8, 32), s(8, 1)),
        lambda: dg.Q4Tensor(u8(8, 32), s(1, 8)), lambda: dg.Q4Tensor(u8(8, 32), s(8, 1), u8(8, 2)),
        lambda: dg.Q4Tensor(u8(8, 32), s(8, 1), s(8, 1)), lambda: dg.Q4Tensor(u8(8, 32), s(8, 1), u8(8, 1).cpu()),
        lambda: dg.Q4Tensor(u8(4, 8, 32)[::2], s(2, 8, 1)), lambda: dg.Q4Tensor(u8(0, 8, 32), s(0, 8, 1)),
        lambda: dg.Q4Tensor(u8(1025, 1, 16), s(1025, 1, 1)),
        lambda: dg.q4_linear(x, u8(8, 32)), lambda: dg.q4_linear(x.half(), q),
        lambda: dg.q4_linear(x.float(), q), lambda: dg.q4_linear(x[:, :32], q),
        lambda: dg.q4_linear(x.cpu(), q), lambda: dg.q4_linear(x.t(), q), lambda: dg.q4_linear(x[0], q),
        lambda: dg.q4_linear(x, q, offsets=off), lambda: dg.q4_linear(x, e),
        lambda: dg.q4_linear(x, e, offsets=off[:2]), lambda: dg.q4_linear(x, e, offsets=off.long()),
        lambda: dg.q4_linear(x, e, offsets=off.cpu()), lambda: dg.q4_linear(x, q, out=s(4, 7)),
        lambda: dg.q4_linear(x, q, out=s(4, 8).half()), lambda: dg.q4_linear(x, q, out=s(4, 8).cpu()),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"call {i} was taken")
    for f, status in [(lambda: dg.q4_linear(s(4, 66)[:, :64], q), dg.GEMM_ERR_MISALIGNED),
                      (lambda: dg.q4_linear(x, q, out=x[:, :8]), dg.GEMM_ERR_INVALID_ARG)]:
        with pytest.raises(dg.GemmError) as err:
            f()
        assert err.value.status == status
    check_device(dg)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows", [4, 40])
def test_long_sums_of_like_terms_keep_their_size(dg, dtype, rows):
    """2^19 terms of one sign: what the tensor cores' truncation takes off a result stays
    below a quarter of what its type rounds (sums in one piece lose 3e-3)."""
    gen = torch.Generator("cuda").manual_seed(16)
    N, K = 64, 1 << 19
    w, _ = _weights(dg, gen, (N,), K, dtype, 128, True)
    w.scales.fill_(2.0 ** -10)
    w.zeros.fill_(0)
    x = (torch.rand((rows, K), generator=gen, device="cuda") * 2.0 ** -9 + 2.0 ** -9).to(TYPES[dtype])
    got = dg.q4_linear(x, w).double()
    check_device(dg)
    k = torch.arange(K, device="cuda")
    want = torch.stack([x.double() @ (((w.codes[n, k // 2].int() >> (4 * (k % 2)).int()) & 15)
                                      .double() * 2.0 ** -10) for n in range(N)], dim=1)
    assert abs(float(((got - want) / want).mean())) <= {"f16": 2.0 ** -13, "bf16": 2.0 ** -10}[dtype]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("N", [1, 3, 66, 129, 131, 257])
@pytest.mark.parametrize("rows,K", [(5, 1100), (16, 4096), (40, 800), (100, 4100)])
def test_last_columns_of_shared_tiles(dg, zeros, rows, K, N):
    """Tiles of few columns whose K a cluster shares, most of which nobody stores or reads,
    one call close behind another: each has the same bits, within the bound."""
    gen = torch.Generator("cuda").manual_seed(rows + N)
    x = _x(gen, rows, K, "bf16")
    w, values = _weights(dg, gen, (N,), K, "bf16", 64, zeros)
    ys = [dg.q4_linear(x, w) for _ in range(20)]
    check_device(dg)
    _check(ys[0], x, values, K, "bf16", rows > 8)
    assert all(torch.equal(y, ys[0]) for y in ys)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows,N,K", [(1, 130, 300), (8, 8192, 2560), (16, 200, 1000)])
def test_few_rows_take_weights_that_fp16_does_not_hold(dg, zeros, rows, N, K):
    """Scales of 20000: integers are multiplied, and only the result has to fit FP16."""
    gen = torch.Generator("cuda").manual_seed(rows)
    w, values = _weights(dg, gen, (N,), K, "f16", 64, zeros)
    values = values / w.scales.double().repeat_interleave(64, dim=1)[:, :K] * 20000
    w.scales.fill_(20000.0)
    x = _x(gen, rows, K, "f16")
    x.mul_(2.0 ** -12)
    y = dg.q4_linear(x, w)
    check_device(dg)
    assert values.abs().max() > 65504 and y.isfinite().all()
    _check(y, x, values, K, "f16", False)
