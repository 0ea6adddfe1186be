"""The root-mean-square norm on the device against float64.

Tolerances: rstd from a float32 sum of H squares, at most H / 32 + 12 additions behind any term, all terms
positive, halved by the root, and a few roundings more: e = (H / 64 + 12) 2^-24 relative.  y takes two products
more.  A dx entry is the sum of rstd d and rstd n mean(d n), the mean with (H / 32 + 12) 2^-24 of the sum of its
terms' magnitudes.  dgamma sums the rows in float32, at most rows additions of 2^-24.
"""
import numpy as np
import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build
from oracle import fp8_block as fb
from rowcheck import EPS32, assert_within, f64

pytestmark = pytest.mark.gpu

BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def run(R, H, xt=BF16, wt=BF16, residual=True, save8=True, y=True, pad=0, eps=1e-5, seed=0, x=None, inplace=False, dres=True):
    g = torch.Generator(device="cuda").manual_seed(seed + R + H)

    def mk(std=1.0, dt=xt):
        t = torch.full((R, H + pad), float("nan"), dtype=dt, device="cuda")
        t[:, :H] = (torch.randn(R, H, generator=g, device="cuda") * std).to(dt)
        return t[:, :H]

    e = lambda dt=xt: torch.full((R, H + pad), 77.0, dtype=dt, device="cuda")  # noqa: E731
    n = B.norm(R, H, x_f32=xt == F32, w_f32=wt == F32, eps=eps, ld_in=H + pad, ld_out=H + pad)
    a = {"x": mk() if x is None else x, "res": mk(0.3) if residual else None, "gamma": (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(wt)}
    a["x0"], a["res0"] = a["x"].clone(), None if a["res"] is None else a["res"].clone()
    hb, yb = (e() if residual else None), (e() if y else None)
    a["h"] = (a["x"] if inplace else hb[:, :H]) if residual else None
    a["y"] = yb[:, :H] if y else None
    a["rstd"] = torch.full((R,), 77.0, device="cuda")
    a["codes"] = torch.full((R, H), 77, dtype=U8, device="cuda") if save8 else None
    a["scales"] = torch.full((-(-H // 128), R), 77.0, device="cuda") if save8 else None
    B.moe_rmsnorm_fwd(n, a["x"], a["res"], a["gamma"], a["h"], a["y"], a["rstd"], a["codes"], a["scales"])
    a["dy"], a["dres"] = mk(0.1), mk(0.1) if dres else None
    dxb = e()
    a["dx"], a["dgamma"] = dxb[:, :H], torch.full((H,), 77.0, dtype=wt, device="cuda")
    ws = torch.full((max(256, B.moe_rmsnorm_workspace_size(n)),), 255, dtype=U8, device="cuda")
    kept = a["x"] if a["h"] is None else a["h"]
    B.moe_rmsnorm_bwd(n, a["dy"], kept, a["rstd"], a["gamma"], a["dres"], a["dx"], a["dgamma"], ws)
    torch.cuda.synchronize()
    for full in ([] if inplace or not residual else [hb]) + ([yb] if y else []) + [dxb]:
        assert bool((full[:, H:] == 77.0).all()), "columns past the row were written"
    a["kept"] = kept
    return a


def check(R, H, **kw):
    a = run(R, H, **kw)
    eps = kw.get("eps", 1e-5)
    h = f64(a["x0"]) + (f64(a["res0"]) if a["res0"] is not None else 0.0)
    gamma = f64(a["gamma"])
    ry, rn, rr = fb.rmsnorm(h, gamma, eps)
    e = (H / 64 + 12) * EPS32
    assert_within(a["rstd"], rr, e * rr, "rstd")
    # the float32 sum x + residual is rounded once itself: relative to the sum, and the sum of squares with it
    esum = 2 * EPS32 if a["res0"] is not None else 0.0
    if a["y"] is not None:
        assert_within(a["y"], ry, (e + 3 * EPS32 + 2 * esum) * np.abs(ry), "y")
    if a["h"] is not None:
        assert_within(a["h"], h, esum * np.abs(h), "h")
    if a["codes"] is not None:
        # of y before its rounding, whose last bits differ: half a step of the code, and the block's scale alike
        c, s = a["codes"].cpu().numpy(), a["scales"].cpu().numpy().astype(np.float64)
        back = fb.rows_back(c, s)
        top = np.abs(np.pad(ry, ((0, 0), (0, -H % 128)))).reshape(R, -1, 128).max(2)
        assert np.allclose(s.T, np.maximum(top, 2.0 ** -100) / 448, rtol=e + 6 * EPS32, atol=0)
        step = np.repeat(s.T, 128, axis=1)[:, :H]
        assert np.all(np.abs(back - ry) <= np.maximum(np.abs(ry) / 16, step * 2.0 ** -10) * (1 + 4 * e + 16 * EPS32) + step * 2.0 ** -20)
    kept, rstd, dy = f64(a["kept"]), f64(a["rstd"]), f64(a["dy"])
    n = kept * rstd[:, None]
    dres = None if a["dres"] is None else f64(a["dres"])
    rdx, rdg = fb.rmsnorm_backward(dy, n, rstd, gamma, dres)
    d = dy * gamma
    mean = (np.abs(d * n)).mean(1, keepdims=True)
    slack = rstd[:, None] * (4 * EPS32 * np.abs(d) + np.abs(n) * mean * (H / 32 + 20) * EPS32) + 2 * EPS32 * np.abs(rdx)
    assert_within(a["dx"], rdx, slack, "dx")
    assert_within(a["dgamma"], rdg, (R + 8) * EPS32 * np.abs(dy * n).sum(0), "dgamma")
    return a


@pytest.mark.parametrize("xt,wt", [(BF16, BF16), (F32, F32), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("R,H", [(1, 1), (1, 8), (3, 100), (5, 127), (2, 128), (7, 129), (33, 256), (9, 1000), (4, 1001), (130, 2048),
                                 (3, 4096), (2, 5001), (3, 8192), (1, 16384), (2, 16383)])
def test_against_float64(R, H, xt, wt):
    check(R, H, xt=xt, wt=wt)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("save8,y", [(False, True), (True, False), (True, True)])
@pytest.mark.parametrize("pad", [0, 8, 3])
def test_what_is_left_out(residual, save8, y, pad):
    for H in (264, 131):
        check(6, H, residual=residual, save8=save8, y=y, pad=pad, dres=residual)


def test_many_rows():
    check(3000, 512)
    check(2500, 257, xt=F32, wt=F32)


def test_h_in_the_place_of_x():
    a, b = run(37, 520, inplace=True), run(37, 520)
    for k in ("h", "y", "rstd", "codes", "scales", "dx", "dgamma"):
        assert torch.equal(a[k], b[k]), k


def test_dx_in_the_place_of_dy_and_dres():
    R, H = 20, 264
    a = run(R, H)
    n = B.norm(R, H)
    ws = torch.zeros(B.moe_rmsnorm_workspace_size(n), dtype=U8, device="cuda")
    for k in ("dy", "dres"):
        t = {"dy": a["dy"].clone(), "dres": a["dres"].clone()}
        B.moe_rmsnorm_bwd(n, t["dy"], a["kept"], a["rstd"], a["gamma"], t["dres"], t[k], a["dgamma"], ws)
        assert torch.equal(t[k], a["dx"])


def test_no_rows():
    n = B.norm(0, 64)
    e = torch.empty(0, 64, dtype=BF16, device="cuda")
    dg, w = torch.full((64,), 77.0, dtype=BF16, device="cuda"), torch.ones(64, dtype=BF16, device="cuda")
    ws = torch.zeros(256, dtype=U8, device="cuda")
    B.moe_rmsnorm_fwd(n, e, None, w, None, e, torch.empty(0, device="cuda"))
    B.moe_rmsnorm_bwd(n, e, e, torch.empty(0, device="cuda"), w, None, e, dg, ws)
    assert not bool(dg.any())


@pytest.mark.parametrize("H", [64, 100, 129, 2048])
@pytest.mark.parametrize("size,xt", [(1e38, BF16), (3e38, F32), (1e-30, BF16), (1e-37, F32), (2.0 ** -130, BF16)])
def test_rows_that_float32_cannot_square(H, size, xt):
    """Their sum of squares is above float32's range or below it; among others that are as usual."""
    g = torch.Generator(device="cuda").manual_seed(H)
    for eps in (0.0, 1e-5):
        x = torch.randn(9, H, generator=g, device="cuda").to(xt)
        x[2::3] = ((torch.rand(3, H, generator=g, device="cuda") * 0.5 + 0.5) * size).to(xt)
        n = B.norm(9, H, x_f32=xt == F32, eps=eps)
        y, rstd = torch.zeros(9, H, dtype=xt, device="cuda"), torch.zeros(9, device="cuda")
        gamma = torch.ones(H, dtype=BF16, device="cuda")
        B.moe_rmsnorm_fwd(n, x, None, gamma, None, y, rstd)
        ry, _, rr = fb.rmsnorm(f64(x), f64(gamma), float(np.float32(eps)))
        assert_within(y, ry, (H / 64 + 16) * EPS32 * np.abs(ry), "y")
        fits = rr < 3.4e38
        # a rstd below 2^-126 keeps fewer bits
        assert np.all(np.abs(f64(rstd) - rr)[fits] <= ((H / 64 + 16) * EPS32 * rr + 2.0 ** -149)[fits])


def test_zero_rows_and_nan():
    x = torch.zeros(4, 136, dtype=BF16, device="cuda")
    x[1, 5], x[2, 7] = float("nan"), float("inf")
    a = run(4, 136, x=x, residual=False, dres=False)
    assert not bool(a["y"][0].any()) and not bool(a["codes"][0].any()) and bool(a["y"][1].isnan().all())
    others = [c for c in range(136) if c != 7]
    assert bool(a["y"][2, 7].isnan()) and not bool(a["y"][2, others].any()) and float(a["rstd"][2]) == 0.0
    assert bool((a["codes"][1] == 0x7F).all()) and bool((a["codes"][2, :128] == 0x7F).all()) and not bool((a["codes"][2, 128:] & 0x7F).any())


def test_reproducible():
    a, b = run(777, 1024), run(777, 1024)
    for k in ("y", "h", "rstd", "codes", "scales", "dx", "dgamma"):
        assert torch.equal(a[k], b[k]), k
