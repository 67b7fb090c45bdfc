"""Cases of the microscaled (MX) operators: a linear layer whose forward
product runs in 4 bits, whose input is kept in 8 bits for the backward pass,
and whose two gradients read the quantised operands directly.

Formats (OCP Microscaling Formats v1.0): a row is cut into blocks of 32
values that share one scale 2^(s - 127), s a byte (E8M0).  MXFP4 elements are
E2M1 (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives), MXINT8 elements are
integers / 64 in +-127/64.  s = floor(log2(max |x| of the block)) - emax + 127
(emax 2 and 0), elements are x / 2^(s - 127) rounded to nearest even and
saturated.

A quantised array of R rows and K columns is held as bytes: codes (R rows,
two MXFP4 codes a byte, the even column low, or one MXINT8 code a byte, row
pitch a multiple of 16) and scales in tiles of 128 rows x 4 blocks: the scale
of row r, block b is byte (r % 32) * 16 + (r % 128 / 32) * 4 + b % 4 of tile
(r / 128) * ceil(blocks / 4) + b / 4, tiles 512 bytes each.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BLOCK = 32


# ------------------------------------------------------------------ cases

def listed():
    return [
        # Keep one token's activations in 8 bits and restore them: the smallest call.
        {"name": "keep 1 token", "op": "roundtrip", "fmt": "mxint8", "type": "bf16",
         "R": 1, "K": 4096, "stored": "N"},
        # Activations of a whole step kept for the backward pass and restored.
        {"name": "keep 8192x8192", "op": "roundtrip", "fmt": "mxint8", "type": "bf16",
         "R": 8192, "K": 8192, "stored": "N"},
        # FP32 master weights stored in x out, odd sizes, quantised for the forward product.
        {"name": "weights 4097x3000", "op": "roundtrip", "fmt": "mxfp4", "type": "f32",
         "R": 4097, "K": 3000, "stored": "T"},
        # Both operands in 4 bits already: the largest product.
        {"name": "product 8192", "op": "product", "type": "bf16", "M": 8192, "N": 8192, "K": 8192},
        # Ragged in every dimension, FP32 result.
        {"name": "product 1000x1030x777", "op": "product", "type": "f32",
         "M": 1000, "N": 1030, "K": 777},
        # One token through a layer: reads the weights once.
        {"name": "linear 1 token", "op": "linear", "type": "bf16", "M": 1, "N": 4096, "K": 4096},
        # A batch of decoding requests.
        {"name": "linear 33 tokens", "op": "linear", "type": "f16", "M": 33, "N": 4096, "K": 4096},
        # A prompt or a training batch.
        {"name": "linear 4096", "op": "linear", "type": "bf16", "M": 4096, "N": 4096, "K": 4096},
        # Gradient of the layer's input, through the 4-bit weights.
        {"name": "grad x 4096", "op": "grad", "fmt": "mxfp4", "stored": "N", "type": "bf16",
         "out": "bf16", "M": 4096, "N": 4096, "K": 4096},
        # The same for a small layer: latency counts.
        {"name": "grad x 256", "op": "grad", "fmt": "mxfp4", "stored": "N", "type": "bf16",
         "out": "bf16", "M": 256, "N": 256, "K": 256},
        # Gradient of the weights from the 8-bit activations of 8192 tokens.
        {"name": "grad w 8192 tokens", "op": "grad", "fmt": "mxint8", "stored": "T",
         "type": "bf16", "out": "f32", "M": 4096, "N": 4096, "K": 8192},
        # The same with ragged sizes.
        {"name": "grad w 777 tokens", "op": "grad", "fmt": "mxint8", "stored": "T", "type": "f16",
         "out": "f16", "M": 1000, "N": 1030, "K": 777},
    ]


def _size(rng, lo, hi):
    """Log-uniform: half of them odd, half a quarter step of a power of two."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 8:
        p = 1 << (v.bit_length() - 1)
        v = max(q for q in (p, p + p // 4, p + 3 * p // 4) if q <= v)
    else:
        v |= 1
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["roundtrip", "product", "linear", "linear", "grad", "grad"])
    if op == "roundtrip":
        return {"op": op, "fmt": rng.choice(["mxfp4", "mxint8"]),
                "type": rng.choice(["f32", "f16", "bf16"]), "R": _size(rng, 1, 8192),
                "K": _size(rng, 32, 8192), "stored": rng.choice(["N", "N", "T"])}
    if op == "product":
        return {"op": op, "type": rng.choice(["f32", "f16", "bf16"]), "M": _size(rng, 128, 8192),
                "N": _size(rng, 128, 8192), "K": _size(rng, 128, 8192)}
    if op == "linear":
        return {"op": op, "type": rng.choice(["f16", "bf16"]), "M": _size(rng, 1, 4096),
                "N": _size(rng, 256, 8192), "K": _size(rng, 256, 8192)}
    t = rng.choice(["f16", "bf16"])
    if rng.random() < 0.5:
        return {"op": op, "fmt": "mxfp4", "stored": "N", "type": t, "out": t,
                "M": _size(rng, 16, 8192), "N": _size(rng, 256, 4096), "K": _size(rng, 256, 4096)}
    return {"op": op, "fmt": "mxint8", "stored": "T", "type": t, "out": rng.choice(["f32", t]),
            "M": _size(rng, 256, 4096), "N": _size(rng, 256, 4096), "K": _size(rng, 16, 8192)}


def _quant_bytes(rows, cols, fmt):
    blocks = -(-cols // BLOCK)
    return rows * (-(-cols // 2) if fmt == "mxfp4" else cols) + rows * blocks


def work(case):
    es = {"f32": 4, "f16": 2, "bf16": 2}
    op, t = case["op"], es[case["type"]]
    if op == "roundtrip":
        n = case["R"] * case["K"]
        return {"bytes": 2 * n * t + 2 * _quant_bytes(case["R"], case["K"], case["fmt"]),
                "flops": 0}
    M, N, K = case["M"], case["N"], case["K"]
    if op == "product":
        b = _quant_bytes(M, K, "mxfp4") + _quant_bytes(N, K, "mxfp4") + M * N * t
    elif op == "linear":
        b = M * K * t + _quant_bytes(N, K, "mxfp4") + M * N * t
    else:
        b = M * K * t + _quant_bytes(K, N, case["fmt"]) + M * N * es[case["out"]]
    return {"bytes": b, "flops": 2 * M * N * K}


# ------------------------------------------------------------------ plain forms (32 bits)

def _blocks(x, fill=0.0):
    """x (R x K) as R x blocks x 32, the last block filled up."""
    R, K = x.shape
    nb = -(-K // BLOCK)
    if nb * BLOCK != K:
        x = torch.nn.functional.pad(x, (0, nb * BLOCK - K), value=fill)
    return x.reshape(R, nb, BLOCK)


def _pow2(e):
    """2^e for integers -126 .. 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantize(x, fmt):
    """Index (0..7 for MXFP4, integer for MXINT8), sign and exponent of x."""
    xb = _blocks(x.float())
    amax = xb.abs().amax(-1, keepdim=True)
    bad = ~(amax <= torch.finfo(torch.float32).max)
    _, e = torch.frexp(torch.where(bad | (amax == 0), torch.ones_like(amax), amax))
    emax = 2 if fmt == "mxfp4" else 0
    e = torch.where(amax == 0, torch.full_like(e, -127), (e - 1 - emax).clamp(-127, 127))
    # Two exact factors: 2^-e itself can be 2^127 times a value near 2^-149.
    half = torch.div(-e, 2, rounding_mode="floor")
    y = torch.where(bad, torch.zeros_like(xb),
                    xb * _pow2(half) * _pow2(-e - half))
    a = y.abs()
    if fmt == "mxfp4":
        idx = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
               + (a >= 3.5) + (a > 5.0))
    else:
        idx = torch.round(a * 64).clamp(max=127).to(torch.uint8)
    return idx, y < 0, torch.where(bad, torch.full_like(e, 128), e).squeeze(-1)


def _values(idx, neg, e, fmt, K):
    """What the codes stand for, in 32 bits (R x K)."""
    if fmt == "mxfp4":
        i = idx.float()   # 0 .5 1 1.5 | 2 3 | 4 6
        v = torch.where(i < 4, i / 2, torch.where(i < 6, i - 2, 2 * i - 8))
    else:
        v = idx.float() / 64
    half = torch.div(e, 2, rounding_mode="floor")
    v = v * _pow2(half).unsqueeze(-1) * _pow2(e - half).unsqueeze(-1)
    v = torch.where(neg, -v, v)
    v = torch.where((e == 128).unsqueeze(-1), torch.full_like(v, math.nan), v)
    return v.reshape(v.shape[0], -1)[:, :K]


def _pack(idx, neg, e, fmt, K):
    """The bytes of a quantised array: codes (R x pitch) and scale tiles."""
    R, nb = e.shape
    if fmt == "mxfp4":
        c = (idx | (neg.to(torch.uint8) << 3)).reshape(R, -1)
        c = c[:, 0::2] | (c[:, 1::2] << 4)
        width = -(-K // 2)
    else:
        c = torch.where(neg, -idx.to(torch.int16), idx.to(torch.int16)).to(torch.int8)
        c = c.view(torch.uint8).reshape(R, -1)
        width = K
    codes = torch.zeros((R, -(-width // 16) * 16), dtype=torch.uint8, device=e.device)
    codes[:, :width] = c[:, :width]
    rt, bt = -(-R // 128), -(-nb // 4)
    s = torch.zeros((rt * 128, bt * 4), dtype=torch.uint8, device=e.device)
    s[:R, :nb] = (e + 127).to(torch.uint8)
    s = s.reshape(rt, 4, 32, bt, 4).permute(0, 3, 2, 1, 4).reshape(-1)
    return codes, s.contiguous()


def _unpack(codes, scales, fmt, K):
    """What a quantised array stands for, in 32 bits."""
    R, nb = codes.shape[0], -(-K // BLOCK)
    rt, bt = -(-R // 128), -(-nb // 4)
    s = scales.reshape(rt, bt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, bt * 4)
    e = s[:R, :nb].to(torch.int32) - 127
    if fmt == "mxfp4":
        c = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(R, -1)[:, :K]
        idx, neg = _blocks(c & 7), _blocks(c) > 7
    else:
        c = _blocks(codes[:, :K].view(torch.int8).to(torch.int16))
        idx, neg = c.abs(), c < 0
    return _values(idx, neg, e, fmt, K)


# ------------------------------------------------------------------ inputs

def _matrix(gen, rows, cols, dtype, scale=1.0):
    """Normal values on the GPU, as a view with rows of a multiple of 16
    bytes, which is what the 16-bit products ask of their operands."""
    step = 16 // dtype.itemsize
    buf = torch.empty((rows, -(-cols // step) * step), dtype=dtype, device="cuda")
    x = buf[:, :cols]
    x.copy_(torch.randn((rows, cols), generator=gen, device="cuda") * scale)
    return x


def _activations(gen, rows, cols, dtype):
    """Normal values with a few columns 20 times as large, as activations have."""
    x = _matrix(gen, rows, cols, dtype)
    loud = torch.rand(cols, generator=gen, device="cuda") < 0.01
    x.mul_(torch.where(loud, 20.0, 1.0).to(dtype))
    return x


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    op, t = case["op"], TYPES[case["type"]]
    s = {"case": dict(case)}
    if op == "roundtrip":
        R, K = case["R"], case["K"]
        if case["stored"] == "T":
            s["x"] = _matrix(gen, K, R, t, 1 / math.sqrt(K)).t()
        else:
            s["x"] = _activations(gen, R, K, t)
        return s
    M, N, K = case["M"], case["N"], case["K"]
    if op == "product":
        a = _activations(gen, M, K, torch.bfloat16)
        s["a"] = _pack(*_quantize(a, "mxfp4"), "mxfp4", K)
    elif op == "linear":
        s["x"] = _activations(gen, M, K, t)
    if op in ("product", "linear"):
        w = _matrix(gen, N, K, torch.float32, 1 / math.sqrt(K))
        s["w"] = _pack(*_quantize(w, "mxfp4"), "mxfp4", K)
        return s
    if case["stored"] == "N":   # dX: dY (M x K) . W (K x N)
        s["a"] = _matrix(gen, M, K, t)
    else:                       # dW: dY^T, dY stored K x M
        s["a"] = _matrix(gen, K, M, t).t()
    b = (_matrix(gen, K, N, torch.float32, 1 / math.sqrt(N)) if case["fmt"] == "mxfp4"
         else _activations(gen, K, N, torch.bfloat16))
    s["b"] = _pack(*_quantize(b, case["fmt"]), case["fmt"], N)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(s):
    case = s["case"]
    op, t = case["op"], TYPES[case["type"]]
    if op == "roundtrip":
        idx, neg, e = _quantize(s["x"], case["fmt"])
        return _values(idx, neg, e, case["fmt"], case["K"]).to(t)
    K = case["K"]
    if op == "grad":
        b = _unpack(*s["b"], case["fmt"], case["N"])
        if t == torch.float16:
            b = b.to(t).float()   # the operand as the product's type holds it
        return torch.matmul(s["a"].float(), b).to(TYPES[case["out"]])
    if op == "product":
        a = _unpack(*s["a"], "mxfp4", K)
    else:
        a = _values(*_quantize(s["x"], "mxfp4"), "mxfp4", K)
    return torch.matmul(a, _unpack(*s["w"], "mxfp4", K).t()).to(t)


def _run_own(s):
    import dense_gemm_major_gb300 as dg
    case = s["case"]
    op, t = case["op"], TYPES[case["type"]]
    if op == "roundtrip":
        return dg.mx_dequantize(dg.mx_quantize(s["x"], case["fmt"]), t)
    if op == "product":
        return dg.mx_matmul(dg.MXTensor(*s["a"], case["K"], "mxfp4"),
                            dg.MXTensor(*s["w"], case["K"], "mxfp4"), dtype=t)
    if op == "linear":
        return dg.mx_linear(s["x"], dg.MXTensor(*s["w"], case["K"], "mxfp4"))
    return dg.mx_grad(s["a"], dg.MXTensor(*s["b"], case["N"], case["fmt"]),
                      dtype=TYPES[case["out"]])


# ------------------------------------------------------------------ 64 bits

def _floor_log2(a):
    """floor(log2(a)) of positive a in 64 bits, from its exponent field."""
    return ((a.view(torch.int64) >> 52) & 0x7FF) - 1023


def _exact_quantized(x, fmt):
    """x after quantisation, from the definition: one power of two for each
    block, one step for each element."""
    R, K = x.shape
    x = x.double()
    out = torch.empty((R, K), dtype=torch.float64, device=x.device)
    for lo in range(0, K, 1024):   # in slices of whole blocks
        part = _blocks(x[:, lo:lo + 1024].contiguous())
        top = part.abs().amax(dim=2, keepdim=True)
        one = torch.ones_like(top)
        scale = _floor_log2(torch.where(top > 0, top, one)) - (2 if fmt == "mxfp4" else 0)
        scale = torch.pow(2.0, scale.clamp(-127, 127).double())
        y = part / scale
        if fmt == "mxfp4":
            big = torch.where(y.abs() >= 1, y.abs(), torch.ones_like(y))
            step = torch.pow(2.0, (_floor_log2(big) - 1).double())
            y = (torch.round(y / step) * step).clamp(-6, 6)
        else:
            y = (torch.round(y * 64) / 64).clamp(-127 / 64, 127 / 64)
        out[:, lo:lo + 1024] = (y * scale).reshape(R, -1)[:, :min(1024, K - lo)]
    return out


def _exact_values(held, fmt, cols):
    """A quantised array's bytes as 64-bit values."""
    codes, scales = held
    rows, nb = codes.shape[0], (cols + 31) // 32
    r = torch.arange(rows, device=codes.device).unsqueeze(1)
    b = torch.arange(nb, device=codes.device).unsqueeze(0)
    at = ((r // 128) * ((nb + 3) // 4) + b // 4) * 512 + (r % 32) * 16 + (r % 128 // 32) * 4 + b % 4
    scale = torch.pow(2.0, scales[at].double() - 127)
    j = torch.arange(cols, device=codes.device)
    if fmt == "mxfp4":
        c = (codes[:, j // 2] >> ((j % 2) * 4).to(torch.uint8)) & 15
        mant, ex = (c & 1).double(), ((c >> 1) & 3).double()
        v = torch.where(ex == 0, mant / 2, (1 + mant / 2) * torch.pow(2.0, ex - 1))
        v = torch.where(c >= 8, -v, v)
    else:
        v = codes[:, :cols].double()
        v = torch.where(v >= 128, v - 256, v) / 64
    return v * scale[:, j // 32]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "roundtrip":
        return _exact_quantized(s["x"], case["fmt"])
    if op == "grad":
        b = _exact_values(s["b"], case["fmt"], case["N"])
        return torch.matmul(s["a"].double(), b)
    w = _exact_values(s["w"], "mxfp4", case["K"])
    a = (_exact_values(s["a"], "mxfp4", case["K"]) if op == "product"
         else _exact_quantized(s["x"], "mxfp4"))
    return torch.matmul(a, w.t())
