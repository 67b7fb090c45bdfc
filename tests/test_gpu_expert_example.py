"""The grouped products and the 4-bit ones together, as examples/expert_layer.py uses
them."""
import os
import sys

import pytest
import torch

from parity import check_device, gpu_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    gpu_lib()
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                    "examples"))
    import expert_layer
    return expert_layer


def _values(q):
    k = torch.arange(q.cols, device="cuda")
    code = (q.codes[..., k // 2].int() >> (4 * (k % 2)).int()) & 15
    return q.scales[..., k // q.group].double() * (code - q.zeros[..., k // q.group].int()).double()


def test_example_runs_and_serves_in_four_bits(example):
    """The 4-bit layer against the same mixture in 64 bits with the weights' values: two
    layers of BF16 results and BF16 weights."""
    first, last, (x, logits, q1, q2), y4 = example.train(steps=3, log=lambda s: None)
    assert first == first and last == last
    w1, w2 = _values(q1), _values(q2)
    for got in y4:
        n = got.shape[0]
        rows, weights, offsets = example.route(logits[:n])
        ids = torch.repeat_interleave(torch.arange(len(w1), device="cuda"), offsets.diff().long())
        h = torch.relu(torch.einsum("ri,roi->ro", x[rows].double(), w1[ids]))
        y = torch.einsum("ri,roi->ro", h, w2[ids]) * weights.double().unsqueeze(1)
        want = torch.zeros((n, y.shape[1]), dtype=torch.float64, device="cuda").index_add(0, rows, y)
        # Each of four roundings (two results, two layers' weights) is off by 2^-8 / sqrt(3)
        # of its value's size on average or less: 4.6e-3 of the whole together.
        assert float((got.double() - want).norm() / want.norm()) <= 1e-2


def test_gradients_of_the_layer(example):
    """Of the input and of both layers' weights, against autograd of the same mixture in
    64 bits, with an expert that no token goes to."""
    gen = torch.Generator("cuda").manual_seed(3)

    def rand(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale
    tokens, experts, width, hidden, out = 75, 5, 64, 104, 40
    logits = rand(tokens, experts)
    logits[:, 3] = -100.0
    w1, w2 = (rand(experts, hidden, width, scale=0.125).bfloat16().float().requires_grad_(),
              rand(experts, out, hidden, scale=0.1).bfloat16().float().requires_grad_())
    x = rand(tokens, width).bfloat16().requires_grad_()
    dy = rand(tokens, out)
    y = example.layer(x, logits, lambda r, o: example.ExpertLinear.apply(r, w1, o),
                      lambda r, o: example.ExpertLinear.apply(r, w2, o))
    (y * dy).sum().backward()
    check_device(example.dg)
    leaves = [t.detach().double().requires_grad_() for t in (x, w1, w2)]

    def product(w):
        def f(rows, offsets):
            ids = torch.repeat_interleave(torch.arange(experts, device="cuda"),
                                          offsets.diff().long())
            return torch.einsum("ri,roi->ro", rows, w[ids])
        return f

    def plain(xx, up, down):
        rows, weights, offsets = example.route(logits)
        h = torch.relu(up(xx[rows], offsets))
        yy = down(h, offsets) * weights.double().unsqueeze(1)
        return torch.zeros((tokens, out), dtype=torch.float64, device="cuda").index_add(0, rows, yy)
    want = plain(leaves[0], product(leaves[1]), product(leaves[2]))
    (want * dy.double()).sum().backward()
    for got, ref in zip((x, w1, w2), leaves):
        assert got.grad.shape == ref.grad.shape
        # At most five BF16 roundings on the way to a gradient, each of 2^-8 / sqrt(3) of
        # its value's size on average or less (5.1e-3 together), and relu's few changes of
        # sign.
        assert float((got.grad.double() - ref.grad).norm() / ref.grad.norm()) <= 2e-2
    assert (w1.grad[3] == 0).all() and (w2.grad[3] == 0).all()
