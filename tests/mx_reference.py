"""Plain 64-bit implementation of the microscaled formats and products, in
numpy, for the tests of the MX operators: written from the format's
definition, sharing nothing with the CUDA path."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
EMAX = {"mxfp4": 2, "mxint8": 0}


def quantize(x, fmt):
    """(codes R x K, as E2M1 codes or integers; scales R x blocks) of a
    float64 array x."""
    x = np.asarray(x, dtype=np.float64)
    R, K = x.shape
    nb = -(-K // 32)
    xp = np.zeros((R, nb * 32))
    xp[:, :K] = x
    xb = xp.reshape(R, nb, 32)
    with np.errstate(invalid="ignore"):
        amax = np.abs(xb).max(axis=2)
    bad = ~np.isfinite(amax)
    _, e = np.frexp(np.where(bad | (amax == 0), 1.0, amax))   # amax = m 2^e, m in [0.5, 1)
    e = np.where(amax == 0, -127, np.clip(e - 1 - EMAX[fmt], -127, 127))
    y = np.where(bad[:, :, None], 0.0, np.ldexp(np.where(bad[:, :, None], 0.0, xb),
                                                -e[:, :, None]))
    a = np.abs(y)
    if fmt == "mxfp4":
        d = np.abs(a[..., None] - E2M1)
        best = d.min(axis=-1, keepdims=True)
        # Nearest; of two equally near neighbours the even code.
        even_first = np.array([0, 2, 4, 6, 1, 3, 5, 7])
        idx = even_first[np.argmax(d[..., even_first] == best, axis=-1)]
        codes = idx + 8 * np.signbit(y)
    else:
        codes = np.sign(y) * np.minimum(np.rint(a * 64), 127)
    scales = np.where(bad, 255, e + 127).astype(np.uint8)
    return codes.reshape(R, nb * 32)[:, :K].astype(np.int64), scales


def values(codes, scales, fmt):
    K = codes.shape[1]
    if fmt == "mxfp4":
        v = E2M1[codes & 7] * np.where(codes >= 8, -1.0, 1.0)
    else:
        v = codes / 64.0
    s = np.repeat(scales.astype(np.int64), 32, axis=1)[:, :K]
    return np.where(s == 255, np.nan, np.ldexp(v, s - 127))


def pack(codes, scales, fmt):
    """The bytes of the codes (R x pitch) and the tiles of scales."""
    R, K = codes.shape
    nb = scales.shape[1]
    if fmt == "mxfp4":
        c = np.zeros((R, (K + 1) // 2 * 2), dtype=np.uint8)
        c[:, :K] = codes
        c = c[:, 0::2] | (c[:, 1::2] << 4)
    else:
        c = codes.astype(np.int8).view(np.uint8)
    out = np.zeros((R, -(-c.shape[1] // 16) * 16), dtype=np.uint8)
    out[:, :c.shape[1]] = c
    T = -(-nb // 4)
    s = np.zeros(-(-R // 128) * T * 512, dtype=np.uint8)
    for b in range(nb):
        r = np.arange(R)
        s[((r // 128) * T + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4] = \
            scales[:, b]
    return out, s


def unpack(codes, scales, K, fmt):
    """codes and scales (as quantize returns them) from their bytes."""
    R = codes.shape[0]
    if fmt == "mxfp4":
        c = np.stack([codes & 15, codes >> 4], axis=-1).reshape(R, -1)[:, :K].astype(np.int64)
    else:
        c = codes[:, :K].view(np.int8).astype(np.int64)
    nb = -(-K // 32)
    T = -(-nb // 4)
    r = np.arange(R)[:, None]
    b = np.arange(nb)[None, :]
    s = scales[((r // 128) * T + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4]
    return c, s


# Unit roundoff of the result types.
UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def bound(ref, total, K, dtype):
    """Largest |error| of a K-term FP32 sum of exact products, rounded to
    dtype: every accumulation step of the tensor cores (16 terms or more)
    may drop up to one unit of the last place of an FP32 partial sum, which
    is at most `total` = sum |a b|; a few more steps for the alignment of a
    step's own terms.  FP16 adds half its smallest subnormal."""
    steps = -(-K // 16) + 16
    sub = 2.0 ** -25 if dtype == "f16" else 0.0
    return steps * 2.0 ** -23 * total + UNIT[dtype] * np.abs(ref) + sub
