"""Oracle of the operators around the expert FFN (test infrastructure only): layer norm, the
gated activation, 8-bit checkpoints of ragged rows, linear layers grouped by expert.

Plain float64 numpy from the formulas.  Pinned by ``tests/test_oracle_block.py``: finite
differences for every gradient, closed forms and special cases for the rest.
"""
from __future__ import annotations

import numpy as np

from . import mxfp8 as mx


def act8(v):
    """Codes [rows][cols] and scale codes [rows][ceil(cols/32)] of v [rows][cols]: the MX rule on
    blocks of 32 consecutive values of a row, the last one short."""
    v = np.asarray(v, dtype=np.float64)
    rows, cols = v.shape
    padded = np.zeros((rows, (cols + 31) // 32 * 32))
    padded[:, :cols] = v
    codes, scales = mx.quantize_blocks(padded, axis=1)
    return codes[:, :cols], scales


def act8_decode(codes, scales):
    rows, cols = codes.shape
    padded = np.zeros((rows, scales.shape[1] * 32), dtype=np.uint8)
    padded[:, :cols] = codes
    return mx.dequantize_blocks(padded, scales, axis=1)[:, :cols]


def layernorm(h, gamma, beta, eps):
    """y, the normalised rows n, mean, rstd."""
    mean = h.mean(axis=1)
    c = h - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(axis=1) + eps)
    n = c * rstd[:, None]
    return n * gamma + beta, n, mean, rstd


def layernorm_backward(dy, n, rstd, gamma, dres=None):
    """dx, dgamma, dbeta from the normalised rows n."""
    d = dy * gamma
    m1 = d.mean(axis=1, keepdims=True)
    m2 = (d * n).mean(axis=1, keepdims=True)
    dx = rstd[:, None] * (d - m1 - n * m2)
    return (dx if dres is None else dx + dres), (dy * n).sum(axis=0), dy.sum(axis=0)


def silu(g):
    return g / (1.0 + np.exp(-g))


def swiglu(g, u, p):
    return silu(g) * u * p[:, None]


def swiglu_backward(g, u, p, da):
    """dg, du, dp."""
    s = 1.0 / (1.0 + np.exp(-g))
    d = da * p[:, None]
    return d * u * s * (1.0 + g * (1.0 - s)), d * g * s, (da * g * s * u).sum(axis=1)


def segments(split_sizes):
    """(expert, first row, end row) of every expert with rows."""
    r = 0
    for e, s in enumerate(split_sizes):
        if s:
            yield e, r, r + int(s)
        r += int(s)


def grouped_linear(x, w, split_sizes):
    y = np.zeros((x.shape[0], w.shape[1]))
    for e, a, b in segments(split_sizes):
        y[a:b] = x[a:b] @ w[e].T
    return y


def grouped_linear_dgrad(dy, w, split_sizes):
    dx = np.zeros((dy.shape[0], w.shape[2]))
    for e, a, b in segments(split_sizes):
        dx[a:b] = dy[a:b] @ w[e]
    return dx


def grouped_linear_wgrad(x, dy, split_sizes):
    dw = np.zeros((len(split_sizes), dy.shape[1], x.shape[1]))
    for e, a, b in segments(split_sizes):
        dw[e] = dy[a:b].T @ x[a:b]
    return dw
