"""GPU tests of the library's per-stream workspaces: captured graphs keep
working after a later call on their stream has needed a larger one, and host
threads may share a stream."""
import threading

import numpy as np
import pytest
import torch

from parity import check_device, gpu_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dg():
    return gpu_lib()


def _capture(step, s):
    """step() as a graph on stream s, after a call that allocates what it needs."""
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs = step()
    return g, outs


def _replays_like_eager(dg, g, outs, step, fills):
    for fill in fills:
        fill()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    check_device(dg)


def test_mx_graph_replays_after_a_larger_call(dg):
    """A layer step whose forward product has its own quantised X and whose
    gradient sums ranges of K, captured; then a larger step on the stream."""
    gen = torch.Generator("cuda").manual_seed(3)

    def rand(rows, cols, dtype=torch.bfloat16):
        return torch.randn((rows, cols), generator=gen, device="cuda").to(dtype)
    w = dg.mx_quantize(rand(640, 768))
    x, dy, wide = rand(80, 768), rand(3000, 256), dg.mx_quantize(rand(3000, 128), "mxint8")

    def step():
        return dg.mx_linear(x, w), dg.mx_grad(dy.t(), wide, dtype=torch.float32)
    s = torch.cuda.Stream()
    g, outs = _capture(step, s)
    big = rand(5000, 768)
    big_dy, big_kept = rand(8192, 512), dg.mx_quantize(rand(8192, 512), "mxint8")
    held = []
    with torch.cuda.stream(s):
        held.append(dg.mx_linear(big, w))
        held.append(dg.mx_grad(big_dy.t(), big_kept, dtype=torch.float32))
    torch.cuda.synchronize()
    # (Whatever the library freed would come back here.)
    held += [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(64)]
    _replays_like_eager(dg, g, outs, step,
                        [lambda: None, lambda: (x.normal_(generator=gen), dy.normal_(generator=gen))])


def test_q4_graph_replays_after_larger_calls(dg):
    """A product whose 4-bit weights go through the workspace in 16 bits, captured; then
    calls that need 150 and 250 MB of it, which a workspace of 256 serves."""
    gen = torch.Generator("cuda").manual_seed(4)

    def weights(N, K):
        return dg.Q4Tensor(torch.randint(0, 256, (N, K // 2), generator=gen, device="cuda",
                                         dtype=torch.uint8),
                           torch.full((N, K // 128), 0.01, device="cuda").bfloat16())
    x = torch.randn((2500, 256), generator=gen, device="cuda").bfloat16()
    w = weights(300, 256)
    big = [weights(N, 4096) for N in (150 * 128, 250 * 128)]
    wide = torch.randn((2100, 4096), generator=gen, device="cuda").bfloat16()
    outs = [torch.empty((2100, q.rows), dtype=torch.bfloat16, device="cuda") for q in big]

    def step():
        return (dg.q4_linear(x, w),)
    s = torch.cuda.Stream()
    g, got = _capture(step, s)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    with torch.cuda.stream(s):
        for q, out in zip(big, outs):
            dg.q4_linear(wide, q, out=out)
        s.synchronize()
    assert free - torch.cuda.mem_get_info()[0] < 320 << 20
    _replays_like_eager(dg, g, got, step, [
        lambda: x.copy_(torch.randn((2500, 256), generator=gen, device="cuda").bfloat16())] * 3)


@pytest.mark.parametrize("shape,larger", [((256, 256, 256), (512, 512, 1024)),    # slices of K
                                          ((2048, 2048, 512), (2048, 4096, 512)),  # cut tiles
                                          ((1000, 1030, 777), (2000, 2062, 1555))])  # re-pitched
def test_sgemm_graph_replays_after_a_larger_call(dg, shape, larger):
    gen = torch.Generator("cuda").manual_seed(4)

    def operands(M, N, K):
        return (torch.randint(-4, 5, (M, K), generator=gen, device="cuda").float(),
                torch.randint(-4, 5, (K, N), generator=gen, device="cuda").float())
    A, B = operands(*shape)
    LA, LB = operands(*larger)
    s = torch.cuda.Stream()
    g, outs = _capture(lambda: (dg.matmul(A, B),), s)
    with torch.cuda.stream(s):
        held = [dg.matmul(LA, LB) for _ in range(2)]
    torch.cuda.synchronize()
    held += [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(64)]
    for seed in range(2):
        A.random_(-4, 5, generator=gen)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        # Sums of small integers: exact in any order.
        assert np.array_equal(outs[0].cpu().numpy(), (A.double() @ B.double()).cpu().numpy())
    check_device(dg)


@pytest.mark.parametrize("per_thread", [False, True])
def test_two_threads_call_on_one_stream(dg, per_thread):
    """Layers of two threads through the C ABI (ctypes lets both run), one of
    them larger at each call: each gets the product of its own rows."""
    gen = torch.Generator("cuda").manual_seed(6)
    w = dg.mx_quantize(torch.randn((256, 512), generator=gen, device="cuda"))
    stream = 2 if per_thread else torch.cuda.Stream().cuda_stream   # 2: cudaStreamPerThread
    calls = 60
    jobs = []
    for t in range(2):
        xs = [torch.randn((70 + (37 * i if t else 0), 512), generator=gen, device="cuda").bfloat16()
              for i in range(calls)]
        ys = [torch.full((x.shape[0], 256), float("nan"), dtype=torch.bfloat16, device="cuda")
              for x in xs]
        jobs.append((xs, ys, [dg.mx_linear(x, w) for x in xs]))
    torch.cuda.synchronize()
    go = threading.Barrier(2)
    status = [None, None]

    def work(t):
        xs, ys, _ = jobs[t]
        go.wait()
        status[t] = [dg.gemm_mx4_linear("bf16", x.shape[0], 256, 512, x.data_ptr(), 512,
                                        w.codes.data_ptr(), w.codes.stride(0), w.scales.data_ptr(),
                                        y.data_ptr(), 256, stream) for x, y in zip(xs, ys)]
    threads = [threading.Thread(target=work, args=(t,)) for t in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    check_device(dg)
    for t, (_, ys, want) in enumerate(jobs):
        assert status[t] == [dg.GEMM_OK] * calls
        for a, b in zip(ys, want):
            assert torch.equal(a, b)


def test_two_threads_call_the_wrappers_on_one_stream(dg):
    """The same through mx_linear and mx_grad, which let other threads run."""
    gen = torch.Generator("cuda").manual_seed(7)
    w = dg.mx_quantize(torch.randn((264, 512), generator=gen, device="cuda"))
    s = torch.cuda.Stream()
    jobs = []
    for t in range(2):
        xs = [torch.randn((70 + 31 * i * (1 + t), 512), generator=gen, device="cuda").bfloat16()
              for i in range(30)]
        jobs.append([(x, dg.mx_linear(x, w)) for x in xs])
        jobs[t] = [(x, y, dg.mx_grad(y, w), torch.empty_like(y), torch.empty_like(x))
                   for x, y in jobs[t]]
    torch.cuda.synchronize()
    go = threading.Barrier(2)

    def work(t):
        go.wait()
        for x, y, _, out, dx in jobs[t]:
            dg.mx_linear(x, w, out=out, stream=s.cuda_stream)
            dg.mx_grad(y, w, out=dx, stream=s.cuda_stream)
    threads = [threading.Thread(target=work, args=(t,)) for t in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    check_device(dg)
    for job in jobs:
        for _, y, want, out, dx in job:
            assert torch.equal(out, y) and torch.equal(dx, want)
