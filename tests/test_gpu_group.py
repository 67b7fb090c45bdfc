"""GPU tests of the products grouped by expert against plain 64-bit products of
each group, within a bound derived from FP32 accumulation and one rounding."""
import threading

import pytest
import torch

import mx_reference as ref
from parity import check_device, gpu_lib

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NAN = float("nan")


@pytest.fixture(scope="module")
def dg():
    return gpu_lib()


def _offsets(sizes, first=0):
    ends = [first]
    for n in sizes:
        ends.append(ends[-1] + n)
    return torch.tensor(ends, dtype=torch.int32, device="cuda")


def _padded(shape, dtype, gen, pad=0, fill=NAN):
    """Normal values in rows of a multiple of 8 elements, `pad` more; the
    padding holds `fill`."""
    pitch = -(-shape[-1] // 8) * 8 + pad
    buf = torch.full((*shape[:-1], pitch), fill, dtype=TYPES[dtype], device="cuda")
    v = buf[..., :shape[-1]]
    v.copy_(torch.randn(shape, generator=gen, device="cuda"))
    return v


def _check(got, want, total, K, dtype):
    """got within the bound of `want` (64 bits; total: sum |a b|)."""
    lim = torch.from_numpy(ref.bound(want.cpu().numpy(), total.cpu().numpy(), K, dtype))
    err = (got.double().cpu() - want.cpu()).abs()
    bad = ~(err <= lim)
    if bad.any():
        at = tuple(int(i) for i in bad.nonzero()[0])
        raise AssertionError((int(bad.sum()), at, float(got[at]), float(want[at]), float(lim[at])))


SIZES = [[1], [0], [0, 0, 1], [5, 0, 3], [256], [257, 31, 33, 0, 1], [16, 15, 17, 32, 128, 129],
         [300, 0, 0, 700], [1] * 40, [0, 513, 0]]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("op", ["N", "T"])
@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("NK", [(1, 1), (33, 70), (256, 128), (300, 517), (129, 64)])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{sum(s)}")
def test_product(dg, dtype, op, out, NK, sizes):
    """All that lies outside the groups is NaN: rows before the first and after the
    last, the operands' padding, the weights of groups without rows; none of it
    shows, and rows and columns of C outside the groups keep what they held."""
    N, K = NK
    gen = torch.Generator("cuda").manual_seed(len(sizes) * 1000 + sum(sizes) + N)
    first, rows = 3, sum(sizes) + 3 + 7
    off = _offsets(sizes, first)
    a = _padded((rows, K), dtype, gen, pad=8)
    a[:first] = NAN
    a[first + sum(sizes):] = NAN
    b = _padded((len(sizes), K, N) if op == "N" else (len(sizes), N, K), dtype, gen)
    for g, n in enumerate(sizes):
        if n == 0:
            b[g] = NAN
    bm = b if op == "N" else b.transpose(1, 2)
    dc = dtype if out == "same" else out
    wide = torch.full((rows, N + 5), 7.0, dtype=TYPES[dc], device="cuda")
    c = wide[:, 2:2 + N]
    assert dg.grouped_matmul(a, bm, off, out=c) is c
    check_device(dg)
    inside = torch.zeros_like(wide, dtype=torch.bool)
    inside[first:first + sum(sizes), 2:2 + N] = True
    assert (wide[~inside] == 7.0).all()
    lo = first
    for g, n in enumerate(sizes):
        x, w = a[lo:lo + n].double(), bm[g].double()
        if n:
            _check(c[lo:lo + n], x @ w, x.abs() @ w.abs(), K, dc)
        lo += n


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("out", ["same", "f32"])
@pytest.mark.parametrize("MN", [(1, 1), (33, 70), (256, 128), (300, 517), (129, 64)])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{sum(s)}")
def test_grad(dg, dtype, out, MN, sizes):
    """As above; a group's neighbours are NaN, one group at a time, so that a row
    too many on either side shows."""
    M, N = MN
    gen = torch.Generator("cuda").manual_seed(len(sizes) * 1000 + sum(sizes) + N)
    first, rows = 3, sum(sizes) + 3 + 7
    off = _offsets(sizes, first)
    dc = dtype if out == "same" else out
    a0, x0 = _padded((rows, M), dtype, gen, pad=8), _padded((rows, N), dtype, gen)
    for parity in (0, 1):
        a, x = _like(a0), _like(x0)
        a[:first], x[:first] = NAN, NAN
        a[first + sum(sizes):], x[first + sum(sizes):] = NAN, NAN
        lo = first
        for g, n in enumerate(sizes):
            if g % 2 != parity:
                a[lo:lo + n], x[lo:lo + n] = NAN, NAN
            lo += n
        wide = torch.full((len(sizes), M + 2, N + 5), 7.0, dtype=TYPES[dc], device="cuda")
        c = wide[:, 1:M + 1, 2:2 + N]
        assert dg.grouped_grad(a, x, off, out=c) is c
        check_device(dg)
        inside = torch.zeros_like(wide, dtype=torch.bool)
        inside[:, 1:M + 1, 2:2 + N] = True
        assert (wide[~inside] == 7.0).all()
        lo = first
        for g, n in enumerate(sizes):
            p, q = a[lo:lo + n].double(), x[lo:lo + n].double()
            if g % 2 == parity or n == 0:
                _check(c[g], p.t() @ q, p.abs().t() @ q.abs(), n, dc)
            else:
                assert c[g].isnan().all()
            lo += n


def _like(v):
    """A copy of a padded view with the same strides."""
    buf = torch.full((v.shape[0], v.stride(0)), NAN, dtype=v.dtype, device="cuda")
    buf[:, :v.shape[1]] = v
    return buf[:, :v.shape[1]]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("op", ["N", "T"])
@pytest.mark.parametrize("case", [([1], 100, 4096), ([64], 256, 1040), ([5, 0, 60, 1], 513, 3000),
                                  ([33], 130, 8200), ([0, 0, 2], 1030, 2056), ([64, 64, 64], 600, 1100)],
                         ids=lambda c: f"{len(c[0])}x{sum(c[0])}-{c[1]}-{c[2]}")
def test_pairs_that_share_long_sums(dg, dtype, out, op, case):
    """Few units of few rows: two or four pairs share K, scaled results too."""
    sizes, N, K = case
    gen = torch.Generator("cuda").manual_seed(N)
    rows = sum(sizes)
    off = _offsets(sizes, 2)
    a = _padded((rows + 5, K), dtype, gen, pad=8)
    a[:2], a[rows + 2:] = NAN, NAN
    b = _padded((len(sizes), K, N) if op == "N" else (len(sizes), N, K), dtype, gen)
    bm = b if op == "N" else b.transpose(1, 2)
    old = torch.randn((rows + 5, N), generator=gen, device="cuda").to(TYPES[out])
    for alpha, beta in ((1.0, 0.0), (0.5, -2.0)):
        c = old.clone()
        dg.grouped_matmul(a, bm, off, out=c, alpha=alpha, beta=beta)
        check_device(dg)
        assert torch.equal(c[:2], old[:2]) and torch.equal(c[rows + 2:], old[rows + 2:])
        lo = 2
        for g, n in enumerate(sizes):
            x, w, o = a[lo:lo + n].double(), bm[g].double(), old[lo:lo + n].double()
            if n:
                _check(c[lo:lo + n], alpha * (x @ w) + beta * o,
                       abs(alpha) * (x.abs() @ w.abs()) + abs(beta) * o.abs(), K + 1, out)
            lo += n
        again = old.clone()
        dg.grouped_matmul(a, bm, off, out=again, alpha=alpha, beta=beta)
        assert torch.equal(again, c)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("case", [([1100], 100, 130), ([1500], 300, 500), ([4000, 0, 1111], 256, 256),
                                  ([1, 5000], 65, 513), ([3001, 3000], 520, 256)],
                         ids=lambda c: f"{len(c[0])}x{sum(c[0])}-{c[1]}-{c[2]}")
def test_pairs_that_share_a_gradient(dg, dtype, out, case):
    """Few units over many rows, with NaN around the groups; and large products of one
    group, whose tiles have more than 64 rows."""
    sizes, M, N = case
    gen = torch.Generator("cuda").manual_seed(M)
    rows = sum(sizes)
    off = _offsets(sizes, 2)
    a, x = _padded((rows + 5, M), dtype, gen, pad=8), _padded((rows + 5, N), dtype, gen)
    a[:2], a[rows + 2:], x[:2], x[rows + 2:] = NAN, NAN, NAN, NAN
    old = torch.randn((len(sizes), M, N), generator=gen, device="cuda").to(TYPES[out])
    for alpha, beta in ((1.0, 0.0), (0.5, 1.0)):
        c = old.clone()
        dg.grouped_grad(a, x, off, out=c, alpha=alpha, beta=beta)
        check_device(dg)
        lo = 2
        for g, n in enumerate(sizes):
            p, q, o = a[lo:lo + n].double(), x[lo:lo + n].double(), old[g].double()
            _check(c[g], alpha * (p.t() @ q) + beta * o,
                   abs(alpha) * (p.abs().t() @ q.abs()) + abs(beta) * o.abs(), n + 1, out)
            lo += n
        again = old.clone()
        dg.grouped_grad(a, x, off, out=again, alpha=alpha, beta=beta)
        assert torch.equal(again, c)
    wide = _padded((rows + 5, 3000), dtype, gen)
    few = _offsets([200, rows - 200] if len(sizes) > 1 else [rows])
    w = _padded((few.numel() - 1, 3000, N), dtype, gen)
    y = dg.grouped_matmul(wide, w, few, dtype=TYPES[out])
    check_device(dg)
    lo = 0
    for g, n in enumerate(few.diff().tolist()):
        p, q = wide[lo:lo + n].double(), w[g].double()
        _check(y[lo:lo + n], p @ q, p.abs() @ q.abs(), 3000, out)
        lo += n


@pytest.mark.parametrize("op", ["N", "T"])
@pytest.mark.parametrize("rows,N,K", [(8, 2500, 1100), (64, 3800, 2100), (300, 1200, 1040),
                                      (8, 9216, 1100), (8, 9700, 1100)])
def test_units_up_to_as_many_as_clusters_run_at_once(dg, op, rows, N, K):
    """10 to 15 units, for clusters of eight CTAs, and around 37, for clusters of four."""
    gen = torch.Generator("cuda").manual_seed(N)
    a = _padded((rows, K), "bf16", gen)
    b = _padded((1, K, N) if op == "N" else (1, N, K), "bf16", gen)
    bm = b if op == "N" else b.transpose(1, 2)
    c = dg.grouped_matmul(a, bm, _offsets([rows]), dtype=torch.float32)
    check_device(dg)
    x, w = a.double(), bm[0].double()
    _check(c, x @ w, x.abs() @ w.abs(), K, "f32")
    assert torch.equal(dg.grouped_matmul(a, bm, _offsets([rows]), dtype=torch.float32), c)
    d = dg.grouped_grad(_padded((1500, 700), "bf16", gen), _padded((1500, N // 3), "bf16", gen),
                        _offsets([1500]))
    check_device(dg)
    assert d.isfinite().all()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N", [400, 833, 1266, 1300, 3000, 3233])
def test_values_of_gradients_up_to_as_many_units_as_clusters_run_at_once(dg, out, N):
    """6 to 15 units, which clusters of eight CTAs share, 18 to 36, of four, and 39, which none
    do."""
    gen = torch.Generator("cuda").manual_seed(N)
    a, x = _padded((1500, 700), "bf16", gen), _padded((1500, N), "bf16", gen)
    d = dg.grouped_grad(a, x, _offsets([1500]), dtype=TYPES[out])
    check_device(dg)
    p, q = a.double(), x.double()
    _check(d[0], p.t() @ q, p.abs().t() @ q.abs(), 1500, out)
    assert torch.equal(dg.grouped_grad(a, x, _offsets([1500]), dtype=TYPES[out]), d)


@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_scaled_and_accumulated(dg, out):
    gen = torch.Generator("cuda").manual_seed(3)
    sizes = [70, 0, 300, 1]
    off = _offsets(sizes)
    a, x = _padded((380, 130), "bf16", gen), _padded((380, 90), "bf16", gen)
    w = _padded((4, 90, 130), "bf16", gen)
    old = torch.randn((380, 90), generator=gen, device="cuda").to(TYPES[out])
    c = old.clone()
    dg.grouped_matmul(a, w.transpose(1, 2), off, out=c, alpha=0.5, beta=-2.0)
    assert torch.equal(c[371:], old[371:])
    lo = 0
    for g, n in enumerate(sizes):
        p, q, o = a[lo:lo + n].double(), w[g].double().t(), old[lo:lo + n].double()
        if n:
            _check(c[lo:lo + n], 0.5 * (p @ q) - 2 * o, 0.5 * (p.abs() @ q.abs()) + 2 * o.abs(),
                   131, out)
        lo += n
    old = torch.randn((4, 130, 90), generator=gen, device="cuda").to(TYPES[out])
    c = old.clone()
    dg.grouped_grad(a, x, off, out=c, alpha=0.5, beta=1.0)
    assert torch.equal(c[1], old[1])                       # an empty group's is kept
    lo = 0
    for g, n in enumerate(sizes):
        p, q, o = a[lo:lo + n].double(), x[lo:lo + n].double(), old[g].double()
        _check(c[g], 0.5 * (p.t() @ q) + o, 0.5 * (p.abs().t() @ q.abs()) + o.abs(), n + 1, out)
        lo += n
    check_device(dg)


def test_products_without_terms(dg):
    """K == 0 or alpha == 0: the groups' part of C is scaled, operands are not read."""
    off = _offsets([3, 0, 2], 1)
    a = torch.full((8, 16), NAN, dtype=torch.bfloat16, device="cuda")
    w = torch.full((3, 16, 24), NAN, dtype=torch.bfloat16, device="cuda")
    for alpha, k in [(0.0, 16), (1.0, 0)]:
        c = torch.full((8, 24), 2.0, device="cuda")
        dg.grouped_matmul(a[:, :k], w[:, :k], off, out=c, alpha=alpha, beta=1.5)
        want = torch.full((8, 24), 2.0, device="cuda")
        want[1:6] = 3.0
        assert torch.equal(c, want)
        dg.grouped_matmul(a[:, :k], w[:, :k], off, out=c, alpha=alpha)
        want[1:6] = 0.0
        assert torch.equal(c, want)
    c = torch.full((3, 16, 24), NAN, device="cuda")
    dg.grouped_grad(a, w[0, :8], off, out=c, alpha=0.0)
    assert (c == 0).all()
    assert (dg.grouped_grad(a[:0], w[0, :0], _offsets([0, 0, 0]), dtype=torch.float32) == 0).all()
    assert dg.grouped_matmul(a[:0], w, _offsets([0, 0, 0])).shape == (0, 24)
    assert dg.grouped_matmul(a, w[:, :, :0], off).shape == (8, 0)
    assert dg.grouped_grad(a, w[0, :8], _offsets([])).shape == (0, 16, 24)
    check_device(dg)


@pytest.mark.parametrize("K,N", [(7, 33), (77, 130), (130, 77)])
def test_contiguous_operands_of_any_width(dg, K, N):
    """Rows that are no multiple of 16 bytes are read from copies."""
    gen = torch.Generator("cuda").manual_seed(K)
    sizes = [40, 0, 300]
    off = _offsets(sizes)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda").bfloat16()
    x, dy, w = rand(340, K), rand(340, N), rand(3, N, K)
    y, dx = dg.grouped_matmul(x, w.transpose(1, 2), off), dg.grouped_matmul(dy, w, off)
    dw = dg.grouped_grad(dy, x, off)
    lo = 0
    for g, n in enumerate(sizes):
        p, q, m = x[lo:lo + n].double(), dy[lo:lo + n].double(), w[g].double()
        if n:
            _check(y[lo:lo + n], p @ m.t(), p.abs() @ m.abs().t(), K, "bf16")
            _check(dx[lo:lo + n], q @ m, q.abs() @ m.abs(), N, "bf16")
        _check(dw[g], q.t() @ p, q.abs().t() @ p.abs(), n, "bf16")
        lo += n
    check_device(dg)


def test_one_matrix_for_all_groups(dg):
    """An expanded B is read where it is, and its gradient is the groups' sum."""
    gen = torch.Generator("cuda").manual_seed(5)
    off = _offsets([100, 0, 57])
    x, w = _padded((157, 64), "f16", gen), _padded((96, 64), "f16", gen)
    got = dg.grouped_matmul(x, w.expand(3, 96, 64).transpose(1, 2), off)
    p, q = x.double(), w.double()
    _check(got, p @ q.t(), p.abs() @ q.abs().t(), 64, "f16")
    check_device(dg)


def test_many_groups(dg):
    """1024 groups, most of them empty or of one row."""
    gen = torch.Generator("cuda").manual_seed(6)
    sizes = [(g * 7919 % 13) // 6 if g != 500 else 400 for g in range(1024)]
    off = _offsets(sizes)
    rows = sum(sizes)
    a, w = _padded((rows, 72), "bf16", gen), _padded((1024, 72, 40), "bf16", gen)
    y = dg.grouped_matmul(a, w, off)
    dw = dg.grouped_grad(a, y, off, dtype=torch.float32)
    ids = torch.repeat_interleave(torch.arange(1024, device="cuda"),
                                  torch.tensor(sizes, device="cuda"))
    p, q = a.double(), w.double()[ids]
    _check(y, torch.bmm(p.unsqueeze(1), q).squeeze(1),
           torch.bmm(p.abs().unsqueeze(1), q.abs()).squeeze(1), 72, "bf16")
    want = torch.zeros((1024, 72, 40), dtype=torch.float64, device="cuda")
    total = torch.zeros_like(want)
    outer = p.unsqueeze(2) * y.double().unsqueeze(1)
    want.index_add_(0, ids, outer)
    total.index_add_(0, ids, outer.abs())
    _check(dw, want, total, 400, "f32")
    check_device(dg)


def test_integers_are_exact(dg):
    """Integers whose sums FP32 holds exactly: every bit, at sizes past a round of
    the grid."""
    gen = torch.Generator("cuda").manual_seed(8)
    sizes = [700, 1, 0, 1500, 33]
    off, rows = _offsets(sizes), sum(sizes)

    def ints(*shape):
        return torch.randint(-2, 3, shape, generator=gen, device="cuda").bfloat16()
    x, dy, w = ints(rows, 1000), ints(rows, 2056), ints(5, 2056, 1000)
    y = dg.grouped_matmul(x, w.transpose(1, 2), off, dtype=torch.float32)
    dx = dg.grouped_matmul(dy, w, off, dtype=torch.float32)
    dw = dg.grouped_grad(dy, x, off, dtype=torch.float32)
    lo = 0
    for g, n in enumerate(sizes):
        p, q, m = x[lo:lo + n].double(), dy[lo:lo + n].double(), w[g].double()
        assert torch.equal(y[lo:lo + n].double(), p @ m.t())
        assert torch.equal(dx[lo:lo + n].double(), q @ m)
        assert torch.equal(dw[g].double(), q.t() @ p)
        lo += n
    check_device(dg)


@pytest.mark.parametrize("raw,meant", [([0, 5, 3, 9], [0, 5, 5, 9]), ([-4, 2, 6, 9], [0, 2, 6, 9]),
                                       ([0, 50, 60, 9], [0, 10, 10, 10]),
                                       ([2 ** 31 - 1, -2 ** 31, 4, 6], [10, 10, 10, 10])])
def test_bad_offsets_stay_inside_and_are_reported(dg, raw, meant):
    gen = torch.Generator("cuda").manual_seed(9)
    a, w = _padded((10, 64), "bf16", gen), _padded((3, 64, 32), "bf16", gen)
    outs = []
    for offsets in (raw, meant):
        c = torch.full((10, 32), 7.0, dtype=torch.bfloat16, device="cuda")
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        dg.grouped_matmul(a, w, off, out=c)
        dw = dg.grouped_grad(a, c, off)
        st, bits = dg.gemm_device_check(torch.cuda.current_stream().cuda_stream)
        assert (st, bits) == ((dg.GEMM_ERR_DEVICE_TIMEOUT, 1 << 9) if offsets is raw
                              else (dg.GEMM_OK, 0))
        outs.append((c, dw))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_long_float32_sums_round_to_nearest(dg):
    """As the microscaled gradients': 32768 terms in sums of 1024 each, a relative
    error of the norm well under 4e-6 (in one piece it is above 2e-5)."""
    gen = torch.Generator("cuda").manual_seed(10)
    a, x = _padded((32768, 128), "bf16", gen), _padded((32768, 96), "bf16", gen)
    got = dg.grouped_grad(a, x, _offsets([32768]), dtype=torch.float32)[0].double()
    want = a.double().t() @ x.double()
    assert float((got - want).norm()) <= 4e-6 * float(want.norm())
    at = a.t().contiguous()                                   # 128 x 32768
    got = dg.grouped_matmul(at, x.contiguous().unsqueeze(0), _offsets([128]),
                            dtype=torch.float32).double()
    assert float((got - want).norm()) <= 4e-6 * float(want.norm())
    check_device(dg)


def _step(dg, x, dy, w, off):
    return (dg.grouped_matmul(x, w.transpose(1, 2), off), dg.grouped_matmul(dy, w, off),
            dg.grouped_grad(dy, x, off, dtype=torch.float32))


def test_gradients_are_those_of_the_layer(dg):
    """Differences of the loss sum(y * dy) in FP64 along random directions."""
    gen = torch.Generator("cuda").manual_seed(11)
    sizes = [33, 0, 90]
    off = _offsets(sizes)
    x, dy, w = _padded((123, 64), "f16", gen), _padded((123, 40), "f16", gen), \
        _padded((3, 40, 64), "f16", gen)
    _, dx, dw = _step(dg, x, dy, w, off)
    ids = torch.repeat_interleave(torch.arange(3, device="cuda"), torch.tensor(sizes, device="cuda"))

    def loss(xx, ww):
        return float((torch.einsum("ri,roi->ro", xx, ww[ids]) * dy.double()).sum())
    for seed in range(3):
        gen.manual_seed(seed)
        ex = torch.randn(x.shape, generator=gen, device="cuda").double()
        ew = torch.randn(w.shape, generator=gen, device="cuda").double()
        xd, wd = x.double(), w.double()
        # (The loss is linear in each: differences of it are exact up to FP64.)
        for got, e, diff in [(dx, ex, loss(xd + ex, wd) - loss(xd - ex, wd)),
                             (dw, ew, loss(xd, wd + ew) - loss(xd, wd - ew))]:
            along = 2 * float((got.double() * e).sum())
            # Each element is off by up to half a unit (2^-11) of itself.
            room = 2 * float((got.double().abs() * e.abs()).sum()) * 2.0 ** -11
            assert abs(along - diff) <= room + 1e-5


def test_graph_replay_with_other_groups(dg):
    """A captured step replays on new values and new offsets with the eager bits."""
    gen = torch.Generator("cuda").manual_seed(12)
    x, dy, w = _padded((600, 320), "bf16", gen), _padded((600, 515), "bf16", gen), \
        _padded((6, 515, 320), "bf16", gen)
    off = _offsets([100] * 6)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        _step(dg, x, dy, w, off)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs = _step(dg, x, dy, w, off)
    for sizes in ([600, 0, 0, 0, 0, 0], [1, 2, 3, 4, 5, 6], [0, 0, 299, 301, 0, 0]):
        off.copy_(_offsets(sizes))
        x.normal_(generator=gen)
        g.replay()
        torch.cuda.synchronize()
        n = sum(sizes)
        want = _step(dg, x, dy, w, off)
        assert torch.equal(outs[0][:n], want[0][:n]) and torch.equal(outs[1][:n], want[1][:n])
        assert torch.equal(outs[2], want[2])
    check_device(dg)


def test_stream_argument_and_the_allocator(dg):
    """Work on a side stream does not get memory that the current stream still
    reads, and its results may be used there."""
    gen = torch.Generator("cuda").manual_seed(13)
    x, dy, w = _padded((512, 1024), "bf16", gen), _padded((512, 1024), "bf16", gen), \
        _padded((4, 1024, 1024), "bf16", gen)
    off = _offsets([128] * 4)
    want = _step(dg, x, dy, w, off)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        busy = [torch.ones_like(t) for t in want for _ in range(2)]
        torch.cuda._sleep(20_000_000)
        sums, sizes = [t.sum(dtype=torch.float64) for t in busy], [t.numel() for t in busy]
        del busy
        s = side.cuda_stream
        got = (dg.grouped_matmul(x, w.transpose(1, 2), off, stream=s),
               dg.grouped_matmul(dy, w, off, stream=s),
               dg.grouped_grad(dy, x, off, dtype=torch.float32, stream=s))
        torch.cuda.current_stream().wait_stream(side)
        copies = [t.clone() for t in got]
        del got
        assert [float(t) for t in sums] == [float(n) for n in sizes]
        for a, b in zip(copies, want):
            assert torch.equal(a, b)
    check_device(dg)


@pytest.mark.parametrize("shared", [False, True], ids=["own streams", "one stream"])
def test_threads_at_once(dg, shared):
    """Calls from several threads whose operands take copies in a workspace, each on its
    own stream and all on one: every thread has its own sizes and results."""
    gen = torch.Generator("cuda").manual_seed(18)
    cases = []
    for i in range(4):
        K, N, off = 501 + 66 * i, 333 - 50 * i, _offsets([40 + i, 0, 300, 7 * i])
        rows = 340 + 8 * i
        x, dy, w = (torch.randn(shape, generator=gen, device="cuda").half()
                    for shape in ((rows, K), (rows, N), (4, N, K)))
        cases.append((x, dy, w, off, _step(dg, x, dy, w, off)))
    one = torch.cuda.Stream()
    streams = [one if shared else torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    wrong = []

    def run(case, stream):
        x, dy, w, off, want = case
        with torch.cuda.stream(stream):
            for _ in range(25):
                got = _step(dg, x, dy, w, off)
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    wrong.append(x.shape)
    threads = [threading.Thread(target=run, args=a) for a in zip(cases, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    check_device(dg)


def test_offsets_past_32_bits(dg):
    """Weights, rows and results whose element offsets pass 2^31 and 2^32."""
    gen = torch.Generator("cuda").manual_seed(14)
    E, N, K = 20, 16384, 16384                              # 5.4e9 weights
    w = torch.zeros((E, N, K), dtype=torch.bfloat16, device="cuda")
    w[E - 1] = torch.randn((N, K), generator=gen, device="cuda").bfloat16()
    w[0] = w[E - 1] + 1
    x = torch.randn((40, K), generator=gen, device="cuda").bfloat16()
    off = _offsets([3] + [0] * (E - 2) + [37])
    y = dg.grouped_matmul(x, w.transpose(1, 2), off)
    dx = dg.grouped_matmul(x, w, off)
    p = x.double()
    for lo, hi, g in ((0, 3, 0), (3, 40, E - 1)):
        m = w[g].double()
        _check(y[lo:hi], p[lo:hi] @ m.t(), p[lo:hi].abs() @ m.abs().t(), K, "bf16")
        _check(dx[lo:hi], p[lo:hi] @ m, p[lo:hi].abs() @ m.abs(), N, "bf16")
    dw = dg.grouped_grad(x, x, off, out=w)
    for lo, hi, g in ((0, 3, 0), (3, 3, 7), (3, 40, E - 1)):
        q = p[lo:hi]
        _check(dw[g, -64:], q[:, -64:].t() @ q, q[:, -64:].abs().t() @ q.abs(), 37, "bf16")
    del w, dw
    rows = 300_000                                          # x 16384 columns: 4.9e9
    a = torch.zeros((rows, K), dtype=torch.bfloat16, device="cuda")
    a[-64:] = torch.randn((64, K), generator=gen, device="cuda").bfloat16()
    m = torch.randn((2, K, 8), generator=gen, device="cuda").bfloat16()
    y = dg.grouped_matmul(a, m, _offsets([40, rows - 40]))
    assert (y[:-64] == 0).all()
    p, q = a[-64:].double(), m[1].double()
    _check(y[-64:], p @ q, p.abs() @ q.abs(), K, "bf16")
    got = dg.grouped_matmul(y, m.transpose(1, 2), _offsets([40, rows - 40]), out=a)
    p = y[-64:].double()
    _check(got[-64:], p @ q.t(), p.abs() @ q.abs().t(), 8, "bf16")
    assert (got[:-64] == 0).all()
    check_device(dg)


def test_refusals_of_the_wrappers(dg):
    x = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((2, 64, 32), dtype=torch.bfloat16, device="cuda")
    off = _offsets([4, 4])
    bad = [
        lambda: dg.grouped_matmul(x.cpu(), w, off), lambda: dg.grouped_matmul(x, w.cpu(), off),
        lambda: dg.grouped_matmul(x, w, off.cpu()), lambda: dg.grouped_matmul(x, w, off.long()),
        lambda: dg.grouped_matmul(x, w, off[:2]), lambda: dg.grouped_matmul(x, w, off[:0]),
        lambda: dg.grouped_matmul(x, w, off.repeat(2)[::2]),
        lambda: dg.grouped_matmul(x, w, off.view(3, 1)),
        lambda: dg.grouped_matmul(x.float(), w.float(), off),
        lambda: dg.grouped_matmul(x.half(), w, off), lambda: dg.grouped_matmul(x, w[0], off),
        lambda: dg.grouped_matmul(x[:, :32], w, off), lambda: dg.grouped_matmul(x[0], w, off),
        lambda: dg.grouped_matmul(x.t(), w[:, :8], off),
        lambda: dg.grouped_matmul(x, w[:, :, ::2], off),
        lambda: dg.grouped_matmul(x, w, off, beta=1.0),
        lambda: dg.grouped_matmul(x, w, off, dtype=torch.float16),
        lambda: dg.grouped_matmul(x, w, off, out=torch.zeros((8, 31), device="cuda")),
        lambda: dg.grouped_matmul(x, w, off, out=torch.zeros((8, 32))),
        lambda: dg.grouped_matmul(x, w.repeat(600, 1, 1)[:1100],
                                  torch.zeros(1101, dtype=torch.int32, device="cuda")),
        lambda: dg.grouped_grad(x, x[:4], off), lambda: dg.grouped_grad(x, x.half(), off),
        lambda: dg.grouped_grad(x, x, off, beta=1.0), lambda: dg.grouped_grad(x, x.t(), off),
        lambda: dg.grouped_grad(x, x, off, out=torch.zeros((2, 64, 63), device="cuda")),
        lambda: dg.grouped_grad(x, x, off, out=torch.zeros((2, 64, 128), device="cuda")[:, :, ::2]),
        lambda: dg.grouped_grad(x, x, off, dtype=torch.float16),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    buf = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
    odd = torch.zeros((8, 66), dtype=torch.bfloat16, device="cuda")[:, :64]
    for f, status in [
            (lambda: dg.grouped_matmul(odd, w, off), dg.GEMM_ERR_MISALIGNED),
            (lambda: dg.grouped_matmul(buf[1:769].view(8, 96)[:, :64], w, off),
             dg.GEMM_ERR_MISALIGNED),
            (lambda: dg.grouped_grad(odd, x, off), dg.GEMM_ERR_MISALIGNED),
            (lambda: dg.grouped_matmul(x, w, off, out=x[:, :32]), dg.GEMM_ERR_INVALID_ARG),
            (lambda: dg.grouped_grad(x[:, :8], x[:, :8], off, out=buf[:128].view(1, 8, 16)
                                     .expand(2, 8, 16)[:, :, :8]), dg.GEMM_ERR_INVALID_ARG)]:
        with pytest.raises(dg.GemmError) as e:
            f()
        assert e.value.status == status
    check_device(dg)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("op", ["N", "T"])
@pytest.mark.parametrize("N", [1, 3, 127, 130, 257, 259, 390])
@pytest.mark.parametrize("rows,K", [(3, 1100), (200, 2050)])
def test_last_columns_of_shared_units(dg, out, op, rows, K, N):
    """Units of few columns whose K pairs of a cluster share, most of which nobody stores or
    reads, one call close behind another: each has the same bits, within the bound.  The
    gradient has the sum over K rows."""
    gen = torch.Generator("cuda").manual_seed(rows + N)
    a = _padded((rows, K), "bf16", gen)
    b = _padded((1, K, N) if op == "N" else (1, N, K), "bf16", gen)
    bm = b if op == "N" else b.transpose(1, 2)
    cs = [dg.grouped_matmul(a, bm, _offsets([rows]), dtype=TYPES[out]) for _ in range(20)]
    check_device(dg)
    x, w = a.double(), bm[0].double()
    _check(cs[0], x @ w, x.abs() @ w.abs(), K, out)
    assert all(torch.equal(c, cs[0]) for c in cs)
    p, q = _padded((K, rows), "bf16", gen), _padded((K, N), "bf16", gen)
    cs = [dg.grouped_grad(p, q, _offsets([K]), dtype=TYPES[out]) for _ in range(20)]
    check_device(dg)
    x, w = p.double(), q.double()
    _check(cs[0][0], x.t() @ w, x.abs().t() @ w.abs(), K, out)
    assert all(torch.equal(c, cs[0]) for c in cs)
