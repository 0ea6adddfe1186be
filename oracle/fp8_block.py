"""Oracle of the root-mean-square norm, the router's balance loss and the 8-bit operands with one float32 scale per
block of 128 (test infrastructure only).

Plain float64 numpy from the formulas; only the quantizer's two quotients and its product are rounded to
float32, as its definition says.  Pinned by ``tests/test_oracle_fp8_block.py``.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
TINY = np.float32(2.0 ** -100)


def _e4m3_table():
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


E4M3 = _e4m3_table()


def encode(v):
    """E4M3 codes of float values, nearest, ties to the even code, saturating at 448."""
    v = np.asarray(v, dtype=np.float64)
    mag = np.abs(v)
    pos = E4M3[:127]
    hi = np.clip(np.searchsorted(pos, mag), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = np.abs(pos[hi] - mag), np.abs(mag - pos[lo])
    pick = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    pick = np.where(mag >= 448.0, 126, pick)
    return (pick + np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def _quantize(blocks, axes):
    """Codes and scales of float32 blocks over the given axes."""
    b = np.asarray(blocks, dtype=np.float32)
    amax = np.abs(b).max(axis=axes, keepdims=True)
    bad = ~np.isfinite(amax)
    top = np.maximum(np.where(bad, np.float32(1), amax), TINY).astype(np.float32)
    up = (np.float32(448.0) / top).astype(np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        codes = np.where(bad, np.uint8(0x7F), encode(np.nan_to_num((b * up).astype(np.float32), nan=0.0, posinf=448.0, neginf=-448.0)))
    return codes, np.where(bad, np.float32(1), (top / np.float32(448.0)).astype(np.float32))


def _pad(v, rows, cols):
    out = np.zeros((-(-v.shape[0] // rows) * rows, -(-v.shape[1] // cols) * cols), dtype=np.float32)
    out[: v.shape[0], : v.shape[1]] = v
    return out


def _cut(v, high, wide):
    p = _pad(np.asarray(v, dtype=np.float32), high, wide)
    codes, scales = _quantize(p.reshape(p.shape[0] // high, high, p.shape[1] // wide, wide), (1, 3))
    return codes.reshape(p.shape)[: v.shape[0], : v.shape[1]], scales[:, 0, :, 0]


def rows8(v):
    """Codes [R][C], scales [ceil(C/128)][R]."""
    c, s = _cut(v, 1, BLOCK)
    return c, np.ascontiguousarray(s.T)


def tiles8(v):
    """Codes [R][C], scales [ceil(R/128)][ceil(C/128)] of one matrix."""
    return _cut(v, BLOCK, BLOCK)


def layout(split):
    """First row of every expert on blocks of 128, and the blocks used."""
    blocks = [-(-n // BLOCK) for n in split]
    first = np.concatenate([[0], np.cumsum(blocks)])
    return first[:-1] * BLOCK, int(first[-1])


def tokens8(v, split, tiles):
    """Codes [B*128][C] and scales [B][C] or (tiles) [B][ceil(C/128)] of the blocks used, every expert's rows on its own."""
    first, used = layout(split)
    C = v.shape[1]
    codes = np.zeros((used * BLOCK, C), dtype=np.uint8)
    scales = np.zeros((used, -(-C // BLOCK) if tiles else C), dtype=np.float32)
    r0 = 0
    for n, f in zip(split, first):
        if n:
            c, s = _cut(v[r0: r0 + n], BLOCK, BLOCK if tiles else 1)
            codes[f: f + n] = c
            scales[f // BLOCK: f // BLOCK + s.shape[0]] = s
        r0 += n
    return codes, scales


def rows_back(codes, scales):
    return E4M3[codes] * np.repeat(scales.astype(np.float64).T, BLOCK, axis=1)[:, : codes.shape[1]]


def tokens_back(codes, scales):
    return E4M3[codes] * np.repeat(scales.astype(np.float64), BLOCK, axis=0)[: codes.shape[0]]


def tiles_back(codes, scales):
    s = np.repeat(np.repeat(scales.astype(np.float64), BLOCK, axis=0), BLOCK, axis=1)
    return E4M3[codes] * s[: codes.shape[0], : codes.shape[1]]


def rmsnorm(h, gamma, eps):
    """y, the normalised rows n, rstd."""
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    n = h * rstd[:, None]
    return n * gamma, n, rstd


def rmsnorm_backward(dy, n, rstd, gamma, dres=None):
    """dx, dgamma from the normalised rows n."""
    d = dy * gamma
    dx = rstd[:, None] * (d - n * (d * n).mean(axis=1, keepdims=True))
    return (dx if dres is None else dx + dres), (dy * n).sum(axis=0)


def balance(logits, idx, alpha, beta, mask=None):
    """counts [E], n, prob [E], (loss, balance, z), dlogits."""
    T, E = logits.shape
    k = idx.shape[1]
    live = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    x = np.where(live[:, None], logits, 0.0)
    top = x.max(axis=1, keepdims=True)
    none = np.isneginf(top)
    e = np.where(none, 0.0, np.exp(x - np.where(none, 0.0, top)))
    z = e.sum(axis=1, keepdims=True)
    s = e / np.where(none, 1.0, z)
    lse = np.where(none, 0.0, np.where(none, 0.0, top) + np.log(np.where(none, 1.0, z)))[:, 0]
    s, lse = np.where(live[:, None], s, 0.0), np.where(live, lse, 0.0)
    n = int(live.sum())
    m = max(n, 1)
    counts = np.bincount(idx[live].ravel(), minlength=E)
    prob = s.sum(axis=0) / m
    bal, zl = E * (counts * prob).sum() / (k * m), (lse ** 2).sum() / m
    f = E * counts / (k * m)
    d = (alpha * s * (f - (s * f).sum(axis=1, keepdims=True)) + 2 * beta * lse[:, None] * s) / m
    return counts, n, prob, (alpha * bal + beta * zl, bal, zl), d
