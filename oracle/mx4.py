"""CPU oracle for the 4-bit microscaled (MXFP4) operators.  TEST
INFRASTRUCTURE, not the product path.

Plain numpy in fp64 from the OCP Microscaling Formats specification v1.0:
blocks of 32 values along a row, shared scale 2^(floor(log2 max|x|) - 2) (at
least 2^-127; NaN where the block holds a NaN or an infinity), elements the
nearest of the E2M1 values 0 0.5 1 1.5 2 3 4 6, ties to the even code,
saturating at 6, zeros keeping their sign.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def blocks(cols: int) -> int:
    return -(-cols // BLOCK)


def quantize(x):
    """(codes uint8 [rows, 16 blocks], scales uint8 [rows, blocks]) of x [rows, cols]."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = blocks(cols)
    v = np.zeros((rows, nb * BLOCK))
    v[:, :cols] = x
    v = v.reshape(rows, nb, BLOCK)
    bad = ~np.isfinite(v).all(-1)
    fin = np.where(bad[..., None], 0.0, v)
    m = np.abs(fin).max(-1) if nb else np.zeros((rows, 0))
    # frexp: m = f 2^e with f in [0.5, 1), so floor(log2 m) = e - 1
    e = np.where(m > 0, np.frexp(m)[1] - 1 - 2, -127)
    byte = np.clip(e + 127, 0, 254)
    a = np.abs(fin) / np.exp2(byte - 127.0)[..., None]
    dist = np.abs(a[..., None] - GRID)
    best = dist.min(-1, keepdims=True)
    # of the nearest values the even code (two neighbours tie at most)
    tie = dist == best
    code = np.where(tie, np.where(np.arange(8) % 2 == 0, 0, 1) * 8 + np.arange(8), 99).argmin(-1)
    code = code + 8 * np.signbit(fin)
    code = np.where(bad[..., None], 0, code).astype(np.uint8).reshape(rows, nb * BLOCK)
    return code[:, 0::2] | (code[:, 1::2] << 4), np.where(bad, 255, byte).astype(np.uint8)


def dequantize(codes, scales, cols: int):
    """fp64 values [rows, cols]."""
    rows = codes.shape[0]
    c = np.stack([codes & 15, codes >> 4], -1).reshape(rows, -1, BLOCK)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127.0))
    v = np.where(c & 8, -1.0, 1.0) * GRID[c & 7] * s[..., None]
    return v.reshape(rows, -1)[:, :cols]


def values(x):
    """The values x [rows, cols] has in MXFP4."""
    return dequantize(*quantize(x), np.asarray(x).shape[1])


def product(a, b, bias=None, relu: bool = False):
    """(act(a b^T + bias), sum |a| |b| + |bias|: the scale of its rounding errors), a [M, K], b [N, K] fp64."""
    with np.errstate(invalid="ignore"):
        c = a @ b.T
        s = np.abs(a) @ np.abs(b).T
        if bias is not None:
            c = c + bias
            s = s + np.abs(bias)
        if relu:
            c = np.where(c < 0.0, 0.0, c)
    return c, s


def linear(x, w, bias=None, relu: bool = False):
    """The layer act(Q(x) Q(w)^T + bias) and its error scale."""
    return product(values(x), values(w), bias, relu)


def linear_backward(dy, x, w, y=None):
    """{name: (gradient, error scale)} of the layer: dx = Q(d) Q(w^T)^T in blocks along the outputs,
    dw = Q(d^T) Q(x^T)^T in blocks along the rows, db = column sums of d; d = dy where y > 0."""
    d = np.asarray(dy, np.float64)
    if y is not None:
        d = np.where(np.asarray(y, np.float64) > 0, d, 0.0)
    x = np.asarray(x, np.float64)
    return {"x": product(values(d), values(np.asarray(w, np.float64).T)),
            "weight": product(values(d.T), values(x.T)),
            "bias": (d.sum(0), np.abs(d).sum(0))}
