"""A two-layer network trained with the microscaled operators.

    python examples/mx_layer.py [steps]

Each linear layer keeps FP32 master weights and quantises them to MXFP4 for
the step; its forward product runs in 4 bits (``mx_linear``), its input is
kept for the backward pass in 8 bits (``mx_quantize`` to MXINT8), and both
gradients are products of the incoming BF16 gradient with a quantised array
(``mx_grad``): that of the input with the 4-bit weights, that of the weights,
in FP32, with the 8-bit input.  Quantisation is passed straight through in
the gradient, as quantised training does.

After training the validation set, quantised once, goes through the first
layer as a product of two quantised arrays (``mx_matmul``).
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_gemm_major_gb300 as dg  # noqa: E402


class MXLinear(torch.autograd.Function):
    """y = x W^T for BF16 x (tokens x in) and FP32 W (out x in)."""

    @staticmethod
    def forward(ctx, x, weight):
        ctx.weight = dg.mx_quantize(weight, "mxfp4")
        ctx.kept = dg.mx_quantize(x, "mxint8")
        return dg.mx_linear(x, ctx.weight)

    @staticmethod
    def backward(ctx, dy):
        dy = dy.contiguous()
        dx = dg.mx_grad(dy, ctx.weight) if ctx.needs_input_grad[0] else None
        dw = dg.mx_grad(dy.t(), ctx.kept, dtype=torch.float32)
        return dx, dw


def train(steps=60, tokens=512, width=256, hidden=512, out=128, seed=0, log=print):
    """Fits a fixed random network of the same shape; returns the first and
    last loss and the validation outputs (4-bit and as in training)."""
    gen = torch.Generator("cuda").manual_seed(seed)

    def rand(rows, cols, scale=1.0):
        return torch.randn((rows, cols), generator=gen, device="cuda") * scale
    t1, t2 = rand(hidden, width, width ** -0.5), rand(out, hidden, hidden ** -0.5)
    w1 = rand(hidden, width, width ** -0.5).requires_grad_()
    w2 = rand(out, hidden, hidden ** -0.5).requires_grad_()
    opt = torch.optim.Adam([w1, w2], lr=3e-3)
    losses = []
    for step in range(steps):
        x = rand(tokens, width).bfloat16()
        with torch.no_grad():
            want = torch.relu(x.float() @ t1.t()) @ t2.t()
        h = torch.relu(MXLinear.apply(x, w1))
        loss = (MXLinear.apply(h, w2).float() - want).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
        if step % 20 == 0 or step == steps - 1:
            log(f"step {step}: loss {losses[-1]:.4f}")
    with torch.no_grad():
        x = rand(tokens, width).bfloat16()
        q1, q2 = dg.mx_quantize(w1, "mxfp4"), dg.mx_quantize(w2, "mxfp4")
        held = dg.mx_quantize(x, "mxfp4")                  # the set, in 4 bits
        h = torch.relu(dg.mx_matmul(held, q1))
        y4 = dg.mx_linear(h, q2)
        y = dg.mx_linear(torch.relu(dg.mx_linear(x, q1)), q2)
        error = (dg.mx_dequantize(held, torch.float32) - x.float()).norm() / x.float().norm()
        log(f"validation set in 4 bits: relative error {float(error):.3f}")
    st, bits = dg.gemm_device_check(torch.cuda.current_stream().cuda_stream)
    if st != dg.GEMM_OK:
        raise dg.GemmError(st, f"device check (fault bits {bits:#x})")
    return losses[0], losses[-1], y4, y


if __name__ == "__main__":
    import __graft_entry__
    __graft_entry__.build()
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 60)
