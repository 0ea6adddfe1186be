"""The oracle of the root-mean-square norm, the balance loss and the blocks of 128 against other ways to the same:
torch's E4M3, brute force, central differences, special cases."""
import numpy as np
import pytest
import torch

from oracle import fp8_block as fb

RNG = np.random.default_rng(5)


def test_encode_is_nearest_with_ties_to_even():
    v = np.concatenate([RNG.normal(size=4000) * 50, fb.E4M3[:127], (fb.E4M3[:126] + fb.E4M3[1:127]) / 2, [0.0, 448.0, 1e9]])
    v = np.concatenate([v, -v]).astype(np.float32)
    ref = torch.tensor(v).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fb.encode(v), ref)
    assert np.array_equal(fb.E4M3[:127], torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("shape", [(1, 1), (3, 128), (130, 129), (257, 300)])
def test_blocks(shape):
    v = (RNG.normal(size=shape) * np.exp(RNG.normal(size=shape))).astype(np.float32)
    c, s = fb.rows8(v)
    assert c.shape == v.shape and s.shape == (-(-shape[1] // 128), shape[0])
    for r in range(shape[0]):
        for b in range(s.shape[0]):
            part = v[r, b * 128: b * 128 + 128]
            assert s[b, r] == np.float32(np.abs(part).max()) / np.float32(448)
    # half a step of E4M3 relative to the value, or of its smallest step
    back = fb.rows_back(c, s)
    step = np.repeat(s.T, 128, axis=1)[:, : shape[1]].astype(np.float64)
    assert np.all(np.abs(back - v) <= np.maximum(np.abs(v) / 16, step * 2.0 ** -10) * (1 + 1e-6))
    c, s = fb.tiles8(v)
    assert s.shape == (-(-shape[0] // 128), -(-shape[1] // 128)) and s[0, 0] == np.abs(v[:128, :128]).max() / np.float32(448)
    assert np.abs(fb.tiles_back(c, s) - v).max() <= np.abs(v).max() / 16 * (1 + 1e-6)


def test_tokens_start_anew_with_every_expert():
    split, v = [3, 0, 129, 128], RNG.normal(size=(260, 70)).astype(np.float32)
    first, used = fb.layout(split)
    assert list(first) == [0, 128, 128, 384] and used == 4
    for tiles in (False, True):
        c, s = fb.tokens8(v, split, tiles)
        back = fb.tiles_back(c, s) if tiles else fb.tokens_back(c, s)
        assert not back[3:128].any() and not back[257:384].any()
        assert np.allclose(back[:3], v[:3], rtol=1 / 16, atol=0.02) and np.allclose(back[128:257], v[3:132], rtol=1 / 16, atol=0.02)
        alone, _ = fb.tokens8(v[3:132], [129], tiles)
        assert np.array_equal(c[128:384], alone)


def test_blocks_that_are_not_finite_or_nothing():
    v = np.zeros((2, 300), dtype=np.float32)
    v[0, 5], v[1, 200] = np.nan, np.inf
    c, s = fb.rows8(v)
    assert np.isnan(fb.E4M3[c[0, :128]]).all() and np.isnan(fb.E4M3[c[1, 128:256]]).all()
    assert not c[0, 128:].any() and s[0, 0] == 1 and s[1, 0] == np.float32(2.0 ** -100) / np.float32(448)


def differences(f, x, g, eps=1e-6):
    """Directional derivatives of f at x against g, in random directions."""
    for _ in range(4):
        d = RNG.normal(size=x.shape)
        num = (f(x + eps * d) - f(x - eps * d)) / (2 * eps)
        assert np.isclose(num, (g * d).sum(), rtol=1e-6, atol=1e-9)


def test_rmsnorm_gradients():
    h, gamma, dy = RNG.normal(size=(5, 33)), RNG.normal(size=33), RNG.normal(size=(5, 33))
    _, n, rstd = fb.rmsnorm(h, gamma, 1e-5)
    dx, dgamma = fb.rmsnorm_backward(dy, n, rstd, gamma)
    differences(lambda x: (fb.rmsnorm(x, gamma, 1e-5)[0] * dy).sum(), h, dx)
    differences(lambda x: (fb.rmsnorm(h, x, 1e-5)[0] * dy).sum(), gamma, dgamma)
    assert np.allclose(fb.rmsnorm(np.full((1, 7), 3.0), np.ones(7), 0.0)[0], 1.0)


@pytest.mark.parametrize("masked", [False, True])
def test_balance_gradient(masked):
    T, E, k = 9, 5, 2
    x = RNG.normal(size=(T, E))
    idx = np.argsort(-x, axis=1)[:, :k]
    mask = (RNG.random(T) < 0.6).astype(np.uint8) if masked else None
    counts, n, prob, loss, d = fb.balance(x, idx, 0.3, 0.2, mask)
    assert counts.sum() == n * k and np.isclose(prob.sum(), 1) and np.isclose(loss[0], 0.3 * loss[1] + 0.2 * loss[2])
    differences(lambda y: fb.balance(y, idx, 0.3, 0.2, mask)[3][0], x, d)
    if masked:
        assert not d[mask == 0].any()


def test_balance_of_even_loads_is_one():
    idx = np.arange(12).reshape(12, 1) % 4
    _, _, _, loss, _ = fb.balance(np.zeros((12, 4)), idx, 1.0, 0.0)
    assert np.isclose(loss[0], 1.0) and np.isclose(loss[2], np.log(4) ** 2)
    _, n, prob, loss, d = fb.balance(np.zeros((12, 4)), idx, 1.0, 1.0, np.zeros(12))
    assert n == 0 and not prob.any() and loss == (0, 0, 0) and not d.any()
