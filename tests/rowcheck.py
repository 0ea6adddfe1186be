"""Elementwise error bounds of the row operators' tests."""
import numpy as np
import torch

EPS32 = 2.0 ** -24


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def unit(t):
    """Half a unit in the last place, relative, of a tensor's type (with the slack of a value that
    the error before the rounding moves into the next binade)."""
    return torch.finfo(t.dtype).eps / 2 * 1.01


def assert_within(got, ref, slack, name):
    """|got - ref| <= one rounding to got's type + slack (array or number); infinities and NaN alike."""
    g = f64(got)
    assert g.shape == ref.shape, (name, g.shape, ref.shape)
    fin = np.isfinite(ref)
    assert np.array_equal(np.isnan(g), np.isnan(ref)), f"{name}: NaN in other places"
    bound = unit(got) * (np.abs(ref) + slack) + slack + 2.0 ** -133     # bf16's subnormal step at the bottom
    bad = fin & ~(np.abs(g - np.where(fin, ref, 0.0)) <= bound)
    if bad.any():
        i = np.unravel_index(int(np.argmax(bad)), bad.shape)
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} beyond the bound, first at {i}: "
                             f"{g[i]!r} for {ref[i]!r}, bound {np.broadcast_to(bound, bad.shape)[i]:.3e}")
