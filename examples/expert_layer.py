"""A mixture-of-experts layer trained with the grouped products, then served with
4-bit weights.

    python examples/expert_layer.py [steps]

A router sends each token to its two best experts.  Tokens are sorted by expert,
and each expert's two linear layers are products over its rows: the forward product
and the input's gradient (``grouped_matmul``), the weights' gradient in FP32
(``grouped_grad``).  The experts' bounds stay on the GPU: nothing waits for them.

After training the experts' weights are rounded to 4 bits with a scale and a zero for
every 64 inputs, and the layer runs on a few tokens and on many (``q4_linear``).
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_major_gb300 as dg  # noqa: E402


class ExpertLinear(torch.autograd.Function):
    """y[rows of g] = x[rows of g] W[g]^T for BF16 x (rows x in, sorted by expert)
    and FP32 W (experts x out x in)."""

    @staticmethod
    def forward(ctx, x, weight, offsets):
        w = weight.to(x.dtype)
        ctx.save_for_backward(x, w, offsets)
        return dg.grouped_matmul(x, w.transpose(1, 2), offsets)

    @staticmethod
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        dx = dg.grouped_matmul(dy, w, offsets) if ctx.needs_input_grad[0] else None
        dw = (dg.grouped_grad(dy, x, offsets, dtype=torch.float32)
              if ctx.needs_input_grad[1] else None)
        return dx, dw, None


def route(logits, best=2):
    """Rows (token, in the order of their experts), their weights and the experts'
    offsets."""
    weights, experts = torch.softmax(logits, dim=1).topk(best, dim=1)
    ids, order = experts.flatten().sort(stable=True)
    offsets = torch.searchsorted(
        ids, torch.arange(logits.shape[1] + 1, device=ids.device)).to(torch.int32)
    return order // best, weights.flatten()[order], offsets


def layer(x, logits, up, down):
    """The mixture's output (tokens x out, FP32); up and down map sorted rows to rows."""
    rows, weights, offsets = route(logits)
    h = torch.relu(up(x[rows], offsets))
    y = down(h, offsets).float() * weights.unsqueeze(1)
    return torch.zeros((x.shape[0], y.shape[1]), device=x.device).index_add(0, rows, y)


def quantise(weight, group=64):
    """FP32 weights (experts x out x in, in a multiple of group) as a Q4Tensor: each
    group from its least to its largest value in 15 steps, the zero among them."""
    E, N, K = weight.shape
    w = weight.detach().view(E, N, K // group, group)
    low, high = w.amin(3).clamp(max=0), w.amax(3).clamp(min=0)
    scale = ((high - low) / 15).clamp(min=1e-8).to(torch.bfloat16)
    s = scale.float().unsqueeze(3)
    zero = torch.round(-low.unsqueeze(3) / s).clamp(0, 15)
    code = (torch.round(w / s) + zero).clamp(0, 15).to(torch.uint8).view(E, N, K)
    return dg.Q4Tensor(code[..., 0::2] | (code[..., 1::2] << 4), scale,
                       zero.squeeze(3).to(torch.uint8), cols=K, group=group)


def train(steps=40, tokens=512, experts=8, width=256, hidden=512, out=128, seed=0, log=print):
    """Fits a fixed random mixture of the same shape; returns the first and last loss,
    and the outputs of the trained layer and of its 4-bit form on the same tokens."""
    gen = torch.Generator("cuda").manual_seed(seed)

    def rand(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale
    router = rand(width, experts)
    t1, t2 = rand(experts, hidden, width, scale=width ** -0.5), \
        rand(experts, out, hidden, scale=hidden ** -0.5)
    w1 = rand(experts, hidden, width, scale=width ** -0.5).requires_grad_()
    w2 = rand(experts, out, hidden, scale=hidden ** -0.5).requires_grad_()
    opt = torch.optim.Adam([w1, w2], lr=3e-3)

    def linear(w):
        return lambda rows, offsets: ExpertLinear.apply(rows, w, offsets)
    losses = []
    for step in range(steps):
        x = rand(tokens, width).bfloat16()
        logits = x.float() @ router
        with torch.no_grad():
            want = layer(x, logits, linear(t1), linear(t2))
        loss = (layer(x, logits, linear(w1), linear(w2)) - want).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
        if step % 20 == 0 or step == steps - 1:
            log(f"step {step}: loss {losses[-1]:.4f}")
    with torch.no_grad():
        q1, q2 = quantise(w1), quantise(w2)
        x = rand(tokens, width).bfloat16()
        logits = x.float() @ router
        y = layer(x, logits, linear(w1), linear(w2))
        y4 = [layer(x[:n], logits[:n], lambda r, o: dg.q4_linear(r, q1, offsets=o),
                    lambda r, o: dg.q4_linear(r, q2, offsets=o)) for n in (1, 7, tokens)]
        log(f"4-bit weights: relative error {float((y4[-1] - y).norm() / y.norm()):.3f}")
    st, bits = dg.gemm_device_check(torch.cuda.current_stream().cuda_stream)
    if st != dg.GEMM_OK:
        raise dg.GemmError(st, f"device check (fault bits {bits:#x})")
    return losses[0], losses[-1], (x, logits, q1, q2), y4


if __name__ == "__main__":
    import __graft_entry__
    __graft_entry__.build()
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 40)
