"""Cases of the grouped products and of the products with 4-bit weights: the
expert layers of a mixture, trained and served.

Groups: rows are sorted by expert, and expert g's are offsets[g] ..
offsets[g + 1] - 1 of them; offsets are 32-bit integers on the GPU, so that a
router's result is used without the host waiting for it.  Rows past the last
offset are padding: nothing of them is read or written.

  product  Y[rows of g] = X[rows of g] . B[g]       B: experts x K x N, stored
           so ("N", an input's gradient through weights that are out x in) or
           as experts x N x K ("T", the forward product with such weights)
  grad     W[g] = A[rows of g]^T . X[rows of g]     the weights' gradient
  q4       Y = X . W^T, W[n, k] = s[n, k / group] * (q[n, k] - z[n, k / group])
           with 4-bit q (two a byte, the even column low), s of X's type, z
           bytes or 8 for all; with experts, each group of rows has its own W
"""
import math
import random

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ cases
#
# rows: rows that belong to groups; pad: rows behind them.  skew: how uneven the
# groups are (0: even); experts without rows come with few rows or much skew.

def listed():
    return [
        # One token sent to two of eight experts, a small layer: the smallest call.
        {"name": "experts 2 rows", "op": "product", "type": "bf16", "stored": "T", "rows": 2,
         "pad": 0, "experts": 8, "N": 1024, "K": 1024, "skew": 0.0},
        # A batch of decoding requests: reads the weights of the experts that it hits.
        {"name": "experts 64 rows", "op": "product", "type": "bf16", "stored": "T", "rows": 64,
         "pad": 0, "experts": 32, "N": 2048, "K": 2048, "skew": 0.2},
        # A prompt or a training batch, few large experts.
        {"name": "experts 8192 rows", "op": "product", "type": "bf16", "stored": "T",
         "rows": 8192, "pad": 0, "experts": 8, "N": 4096, "K": 4096, "skew": 0.1},
        # Ragged in every dimension, with padding rows behind the last group.
        {"name": "experts 4097 rows", "op": "product", "type": "f16", "stored": "T",
         "rows": 4097, "pad": 103, "experts": 16, "N": 1030, "K": 777, "skew": 1.0},
        # Gradient of the input of many small experts, through weights stored out x in.
        {"name": "grad x 8192 rows", "op": "product", "type": "bf16", "stored": "N",
         "rows": 8192, "pad": 0, "experts": 32, "N": 1024, "K": 4096, "skew": 0.2},
        # Gradient of the weights of the large experts, as a training step keeps it.
        {"name": "grad w 8192 rows", "op": "grad", "type": "bf16", "out": "f32", "rows": 8192,
         "pad": 0, "experts": 8, "N": 4096, "K": 4096, "skew": 0.1},
        # The same with ragged sizes and experts without rows.
        {"name": "grad w 777 rows", "op": "grad", "type": "f16", "out": "f16", "rows": 777,
         "pad": 23, "experts": 16, "N": 1000, "K": 1030, "skew": 8.0},
        # One token through a layer with 4-bit weights.
        {"name": "q4 1 token", "op": "q4", "type": "bf16", "rows": 1, "pad": 0, "experts": 0,
         "N": 4096, "K": 4096, "group": 128, "zeros": False, "skew": 0.0},
        # A few requests at once, the largest layer, scales for every 64 values.
        {"name": "q4 7 tokens 8192", "op": "q4", "type": "f16", "rows": 7, "pad": 0,
         "experts": 0, "N": 8192, "K": 8192, "group": 64, "zeros": True, "skew": 0.0},
        # A batch of decoding requests.
        {"name": "q4 33 tokens", "op": "q4", "type": "bf16", "rows": 33, "pad": 0, "experts": 0,
         "N": 4096, "K": 4096, "group": 128, "zeros": True, "skew": 0.0},
        # Eight tokens sent to two experts each, out of 32 with 4-bit weights.
        {"name": "q4 experts 16 rows", "op": "q4", "type": "bf16", "rows": 16, "pad": 4,
         "experts": 32, "N": 2048, "K": 2048, "group": 32, "zeros": True, "skew": 0.5},
        # A prompt through the same layer.
        {"name": "q4 4096 tokens", "op": "q4", "type": "bf16", "rows": 4096, "pad": 0,
         "experts": 0, "N": 4096, "K": 4096, "group": 128, "zeros": True, "skew": 0.0},
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
    op = rng.choice(["product", "product", "grad", "q4", "q4"])
    case = {"op": op, "type": rng.choice(["f16", "bf16"]), "rows": _size(rng, 1, 8192),
            "pad": rng.choice([0, 0, rng.randint(1, 200)]),
            "skew": round(rng.choice([0.0, rng.uniform(0.0, 1.0), rng.uniform(1.0, 8.0)]), 3)}
    N, K = _size(rng, 64, 4096), _size(rng, 64, 4096)
    experts = _size(rng, 1, 128)
    if op == "q4":
        case["rows"] = _size(rng, 1, rng.choice([16, 64, 4096]))
        case["group"] = rng.choice([32, 64, 128])
        case["zeros"] = rng.random() < 0.5
        if rng.random() < 0.5:
            case["pad"] = experts = 0
            N, K = 2 * N, 2 * K
    elif op == "product":
        case["stored"] = rng.choice(["N", "T"])
    else:
        case["out"] = rng.choice(["f32", case["type"]])
    # At most 2^27 weights (the largest listed layer), and 2^36 products in all.
    while max(experts, 1) * N * K > 1 << 27 and experts > 1:
        experts -= 1
    while case["rows"] * N * K > 1 << 36:
        case["rows"] = case["rows"] // 2 | 1
    case.update(experts=experts, N=N, K=K)
    return case


def _group_sizes(case):
    """Rows of the groups, largest first: shares 1 / (1 + skew * g) of them."""
    E = max(case["experts"], 1)
    share = [1.0 / (1.0 + case["skew"] * g) for g in range(E)]
    total, sizes, used = sum(share), [], 0
    for g in range(E):
        sizes.append(int(case["rows"] * share[g] / total))
        used += sizes[-1]
    for i in range(case["rows"] - used):   # what rounding down left
        sizes[i % E] += 1
    return sizes


def work(case):
    R, N, K, t = case["rows"], case["N"], case["K"], BYTES[case["type"]]
    E, hit = max(case["experts"], 1), sum(1 for s in _group_sizes(case) if s)
    offsets = 4 * (case["experts"] + 1) if case["experts"] else 0
    if case["op"] == "product":
        b = R * (K + N) * t + hit * N * K * t
    elif case["op"] == "grad":
        b = R * (K + N) * t + E * N * K * BYTES[case["out"]]
    else:
        per_row = (K + 1) // 2 + -(-K // case["group"]) * (t + (1 if case["zeros"] else 0))
        b = R * (K + N) * t + hit * N * per_row
    return {"bytes": b + offsets, "flops": 2 * R * N * K}


# ------------------------------------------------------------------ inputs

def _array(gen, shape, dtype, scale=1.0):
    """Normal values on the GPU, as a view with rows of a multiple of 16
    bytes, which is what the 16-bit products ask of their operands."""
    step = 16 // dtype.itemsize
    cols = shape[-1]
    buf = torch.empty((*shape[:-1], -(-cols // step) * step), dtype=dtype, device="cuda")
    x = buf[..., :cols]
    if x.dim() == 3:   # one expert at a time: the 32-bit values of all are large
        for part in x:
            part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * scale)
    else:
        x.copy_(torch.randn(shape, generator=gen, device="cuda") * scale)
    return x


def _activations(gen, rows, cols, dtype):
    """Normal values with a few columns 20 times as large, as activations have."""
    x = _array(gen, (rows, cols), dtype)
    loud = torch.rand(cols, generator=gen, device="cuda") < 0.01
    x.mul_(torch.where(loud, 20.0, 1.0).to(dtype))
    return x


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(int(seed))
    op, t = case["op"], TYPES[case["type"]]
    R, E, N, K = case["rows"] + case["pad"], case["experts"], case["N"], case["K"]
    s = {"case": dict(case), "offsets": None}
    if E:
        sizes = _group_sizes(case)
        random.Random(int(seed)).shuffle(sizes)   # which expert is popular is data
        ends = [0]
        for n in sizes:
            ends.append(ends[-1] + n)
        s["ends"] = ends   # what a program in plain torch would have to know on the host
        s["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
    if op == "product":
        s["x"] = (_activations(gen, R, K, t) if case["stored"] == "T" else
                  _array(gen, (R, K), t))
        shape = (E, N, K) if case["stored"] == "T" else (E, K, N)
        s["w"] = _array(gen, shape, t, 1 / math.sqrt(K))
    elif op == "grad":
        s["dy"] = _array(gen, (R, N), t)
        s["x"] = _activations(gen, R, K, t)
    else:
        s["x"] = _activations(gen, R, K, t)
        lead = (E, N) if E else (N,)
        groups = -(-K // case["group"])
        pitch = -(-((K + 1) // 2) // 16) * 16
        s["codes"] = torch.randint(0, 256, (*lead, pitch), generator=gen, device="cuda",
                                   dtype=torch.uint8)
        # (Steps of a quarter of the weights' deviation, as 4 bits take them.)
        u = torch.rand((*lead, groups), generator=gen, device="cuda")
        s["scales"] = ((0.15 + 0.2 * u) / math.sqrt(K)).to(t)
        s["zeros"] = None
        if case["zeros"]:
            s["zeros"] = torch.randint(5, 12, (*lead, groups), generator=gen, device="cuda",
                                       dtype=torch.uint8)
    if op != "grad":
        # The caller's buffer, whose padding rows keep what they hold.
        s["out"] = _array(gen, (R, N), t)
    if own and op == "q4":
        import dense_gemm_major_gb300 as dg
        s["q"] = dg.Q4Tensor(s["codes"], s["scales"], s["zeros"], cols=K, group=case["group"])
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _q4_values(codes, scales, zeros, K, group):
    """4-bit weights as 32-bit values."""
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)[..., :K].float()
    each = torch.arange(K, device=codes.device) // group
    z = 8.0 if zeros is None else zeros.float()[..., each]
    return (q - z) * scales.float()[..., each]


def _run_plain(s):
    case = s["case"]
    op, E = case["op"], case["experts"]
    if op == "grad":
        t = TYPES[case["out"]]
        w = torch.empty((E, case["N"], case["K"]), dtype=t, device=s["x"].device)
        for g in range(E):
            a, b = s["ends"][g], s["ends"][g + 1]
            w[g] = torch.matmul(s["dy"][a:b].float().t(), s["x"][a:b].float()).to(t)
        return w
    out, t = s["out"], TYPES[case["type"]]
    if op == "q4" and not E:
        w = _q4_values(s["codes"], s["scales"], s["zeros"], case["K"], case["group"])
        rows = case["rows"]
        out[:rows] = torch.matmul(s["x"][:rows].float(), w.t()).to(t)
        return out
    for g in range(E):
        a, b = s["ends"][g], s["ends"][g + 1]
        if a == b:
            continue
        if op == "product":
            w = s["w"][g].float()
            w = w.t() if case["stored"] == "T" else w
        else:
            w = _q4_values(s["codes"][g], s["scales"][g],
                           None if s["zeros"] is None else s["zeros"][g], case["K"],
                           case["group"]).t()
        out[a:b] = torch.matmul(s["x"][a:b].float(), w).to(t)
    return out


def _run_own(s):
    import dense_gemm_major_gb300 as dg
    case = s["case"]
    if case["op"] == "product":
        w = s["w"].transpose(1, 2) if case["stored"] == "T" else s["w"]
        return dg.grouped_matmul(s["x"], w, s["offsets"], out=s["out"])
    if case["op"] == "grad":
        return dg.grouped_grad(s["dy"], s["x"], s["offsets"], dtype=TYPES[case["out"]])
    return dg.q4_linear(s["x"], s["q"], offsets=s["offsets"], out=s["out"])


# ------------------------------------------------------------------ 64 bits

def _weights64(s, g):
    """Expert g's weights (K x N) in 64 bits (g None: the only ones)."""
    case = s["case"]
    if case["op"] == "product":
        w = s["w"][g].to(torch.float64)
        return w.transpose(0, 1) if case["stored"] == "T" else w
    pick = (lambda a: a) if g is None else (lambda a: a[g])
    codes, scales = pick(s["codes"]), pick(s["scales"])
    k = torch.arange(case["K"], device=codes.device)
    q = (codes[:, k // 2].to(torch.int32) >> (4 * (k % 2)).to(torch.int32)) & 15
    z = 8 if s["zeros"] is None else pick(s["zeros"])[:, k // case["group"]].to(torch.int32)
    w = scales[:, k // case["group"]].double() * (q - z).double()
    return w.transpose(0, 1)


def exact(case, seed):
    s = prepare(case, seed)
    E, N, K = case["experts"], case["N"], case["K"]
    x = s["x"]
    if case["op"] == "grad":
        w = torch.zeros((E, N, K), dtype=torch.float64, device=x.device)
        for g in range(E):
            rows = slice(s["ends"][g], s["ends"][g + 1])
            w[g] = s["dy"][rows].double().transpose(0, 1) @ x[rows].double()
        return w
    y = s["out"].double()
    if not E:
        y[:case["rows"]] = x[:case["rows"]].double() @ _weights64(s, None)
        return y
    for g in range(E):
        rows = slice(s["ends"][g], s["ends"][g + 1])
        if rows.stop > rows.start:
            y[rows] = x[rows].double() @ _weights64(s, g)
    return y
