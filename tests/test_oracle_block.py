"""Pins of the oracle of the operators around the expert FFN: finite differences for the
gradients, closed forms and special cases for the rest."""
import numpy as np
import pytest
import torch

from oracle import block as bl
from oracle import mxfp8 as mx


def central(f, x, h=1e-6):
    """Gradient of the scalar f at x by central differences (float64: error about 1e-9)."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("rows,H", [(1, 1), (3, 7), (2, 32)])
def test_layernorm_gradients(rows, H):
    r = np.random.default_rng(1)
    x, dy, gamma, beta = r.normal(size=(rows, H)), r.normal(size=(rows, H)), r.normal(size=H), r.normal(size=H)
    eps = 1e-2
    loss = lambda x, g, b: float((bl.layernorm(x, g, b, eps)[0] * dy).sum())  # noqa: E731
    _, n, _, rstd = bl.layernorm(x, gamma, beta, eps)
    dx, dg, db = bl.layernorm_backward(dy, n, rstd, gamma)
    assert np.allclose(dx, central(lambda v: loss(v, gamma, beta), x), atol=1e-6)
    assert np.allclose(dg, central(lambda v: loss(x, v, beta), gamma), atol=1e-6)
    assert np.allclose(db, central(lambda v: loss(x, gamma, v), beta), atol=1e-6)
    dres = r.normal(size=(rows, H))
    assert np.allclose(bl.layernorm_backward(dy, n, rstd, gamma, dres)[0], dx + dres)


def test_layernorm_matches_torch_in_float64():
    r = np.random.default_rng(2)
    x, gamma, beta = r.normal(size=(5, 40)) * 3 + 1, r.normal(size=40), r.normal(size=40)
    y = bl.layernorm(x, gamma, beta, 1e-5)[0]
    t = torch.nn.functional.layer_norm(torch.from_numpy(x), (40,), torch.from_numpy(gamma), torch.from_numpy(beta), 1e-5)
    assert np.allclose(y, t.numpy(), rtol=1e-12, atol=1e-12)


def test_swiglu_gradients():
    r = np.random.default_rng(3)
    g, u, p, da = r.normal(size=(3, 5)) * 2, r.normal(size=(3, 5)), r.random(3), r.normal(size=(3, 5))
    dg, du, dp = bl.swiglu_backward(g, u, p, da)
    loss = lambda g, u, p: float((bl.swiglu(g, u, p) * da).sum())  # noqa: E731
    assert np.allclose(dg, central(lambda v: loss(v, u, p), g), atol=1e-7)
    assert np.allclose(du, central(lambda v: loss(g, v, p), u), atol=1e-7)
    assert np.allclose(dp, central(lambda v: loss(g, u, v), p), atol=1e-7)


@pytest.mark.parametrize("split", [[2, 0, 3], [0, 0, 5], [5], [1, 1, 3]])
def test_grouped_linear_gradients(split):
    r = np.random.default_rng(4)
    x, w, dy = r.normal(size=(5, 4)), r.normal(size=(len(split), 3, 4)), r.normal(size=(5, 3))
    loss = lambda x, w: float((bl.grouped_linear(x, w, split) * dy).sum())  # noqa: E731
    assert np.allclose(bl.grouped_linear_dgrad(dy, w, split), central(lambda v: loss(v, w), x), atol=1e-7)
    assert np.allclose(bl.grouped_linear_wgrad(x, dy, split), central(lambda v: loss(x, v), w), atol=1e-7)


def test_grouped_linear_is_each_row_by_its_expert():
    r = np.random.default_rng(5)
    split = [3, 0, 1, 2]
    x, w = r.normal(size=(8, 6)), r.normal(size=(4, 5, 6))
    owner = np.repeat(np.arange(4), split)
    y = bl.grouped_linear(x, w, split)
    for i, e in enumerate(owner):
        assert np.allclose(y[i], w[e] @ x[i])
    assert not y[6:].any()                                   # rows past the sum


@pytest.mark.parametrize("cols", [1, 31, 32, 33, 70])
def test_act8_blocks(cols):
    """A short block behaves as the same values followed by zeros; a round trip keeps every value
    within half a step of E4M3 (2^-4 of it, or 2^-10 of the block's scale)."""
    r = np.random.default_rng(cols)
    v = r.normal(size=(6, cols)) * np.exp(r.normal(size=(6, 1)) * 3)
    codes, scales = bl.act8(v)
    assert codes.shape == v.shape and scales.shape == (6, (cols + 31) // 32)
    back = bl.act8_decode(codes, scales)
    scale = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, axis=1)[:, :cols]
    assert np.all(np.abs(back - v) <= np.maximum(np.abs(v) / 16, scale / 1024) * (1 + 1e-12))
    full = np.zeros((6, (cols + 31) // 32 * 32))
    full[:, :cols] = v
    assert np.array_equal(codes, mx.quantize_blocks(full, axis=1)[0][:, :cols])
    # what is kept is kept again unchanged (the values: a maximum that was rounded down to half
    # the range takes the next smaller scale, and then other codes)
    assert np.array_equal(bl.act8_decode(*bl.act8(back)), back)
