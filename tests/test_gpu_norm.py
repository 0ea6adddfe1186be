"""Layer norm on the GPU, forward and backward, against float64.

Bounds: one rounding to the output's type, plus float32 sums.  A sum over H values in the kernel's
tree has fewer than 64 additions behind any term for H <= 16384 (16 per thread, 5 + 5 shuffles), so
its error is below 64 * 2^-24 of the sum of magnitudes; the same holds, with fewer than 512
additions, for the weights' gradients at these row counts.
"""
import numpy as np
import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build
from oracle import block as bl
from rowcheck import EPS32, assert_within, f64

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def wide(rows, H, ld, dtype, g, std=1.0, mean=0.0):
    """A [rows][H] view at row pitch ld whose unused columns hold NaN."""
    t = torch.full((rows, ld), float("nan"), dtype=dtype, device="cuda")
    t[:, :H] = (torch.randn(rows, H, generator=g, device="cuda") * std + mean).to(dtype)
    return t[:, :H]


def out_like(rows, H, ld, dtype):
    t = torch.full((rows, ld), 77.0, dtype=dtype, device="cuda")
    return t, t[:, :H]


CASES = [
    # rows, H, x f32, w f32, residual, act8, ld_in - H, ld_out - H
    (1, 1, False, False, False, False, 0, 0),
    (1, 1024, False, False, False, True, 0, 0),
    (3, 8, False, True, True, True, 0, 0),
    (5, 40, False, False, True, True, 8, 16),
    (7, 33, False, False, True, True, 0, 0),
    (9, 31, True, True, False, True, 0, 3),
    (130, 513, True, False, True, True, 1, 0),
    (65, 2048, False, False, True, True, 0, 0),
    (1237, 1001, True, True, False, False, 0, 0),
    (700, 768, False, True, True, False, 8, 0),
    (40, 4096, True, True, True, True, 0, 0),
    (33, 4104, False, False, False, True, 0, 0),
    (17, 4097, False, False, True, True, 0, 0),
    (9, 16384, False, False, True, True, 0, 0),
    (6, 16384, True, True, False, False, 4, 4),
    (5, 16383, True, True, False, True, 0, 0),
    (3000, 264, False, False, True, True, 0, 0),
]


@pytest.mark.parametrize("rows,H,xf,wf,residual,act8,pin,pout", CASES)
def test_layernorm(rows, H, xf, wf, residual, act8, pin, pout):
    g = torch.Generator(device="cuda").manual_seed(rows * 7 + H)
    t, wt = torch.float32 if xf else torch.bfloat16, torch.float32 if wf else torch.bfloat16
    n = B.norm(rows, H, x_f32=xf, w_f32=wf, eps=EPS, ld_in=H + pin, ld_out=H + pout)
    x = wide(rows, H, H + pin, t, g, 2.0, 0.7)
    res = wide(rows, H, H + pin, t, g, 0.5) if residual else None
    gamma = (torch.randn(H, generator=g, device="cuda") * 0.2 + 1).to(wt)
    beta = (torch.randn(H, generator=g, device="cuda") * 0.2).to(wt)
    yb, y = out_like(rows, H, H + pout, t)
    hb, h = out_like(rows, H, H + pout, t) if residual else (None, None)
    mean = torch.empty(rows, device="cuda")
    rstd = torch.empty(rows, device="cuda")
    codes = torch.zeros(rows, H, dtype=torch.uint8, device="cuda") if act8 else None
    scales = torch.zeros(rows, (H + 31) // 32, dtype=torch.uint8, device="cuda") if act8 else None
    B.moe_layernorm_fwd(n, x, res, gamma, beta, h, y, mean, rstd, codes, scales)
    torch.cuda.synchronize()

    x64 = f64(x) + (f64(res) if residual else 0.0)
    ry, rn, rmean, rrstd = bl.layernorm(x64, f64(gamma), f64(beta), EPS)
    # the centred value h - mu: its own rounding and that of mu, whose error is a row sum's
    cen = (np.abs(x64) + np.abs(x64).mean(1, keepdims=True)) * rrstd[:, None]
    # rstd: the centred values' errors enter the variance to first order through |n|
    rel = 64 * EPS32 * (1 + 2 * (np.abs(rn) * cen).mean(1, keepdims=True))
    en = 64 * EPS32 * cen + np.abs(rn) * rel
    assert_within(y, ry, en * np.abs(f64(gamma)) + 4 * EPS32 * np.abs(f64(beta)), "y")
    assert_within(mean, rmean, 64 * EPS32 * np.abs(x64).mean(1), "mean")
    assert_within(rstd, rrstd, rrstd * rel[:, 0], "rstd")
    if residual:
        assert_within(h, x64, EPS32 * (np.abs(f64(x)) + np.abs(f64(res))), "h")
    for full in (yb, hb):
        if full is not None and pout:
            assert bool((full[:, H:] == 77.0).all()), "columns past the row were written"
    if act8:
        back = bl.act8_decode(codes.cpu().numpy(), scales.cpu().numpy())
        step = np.repeat(np.ldexp(1.0, scales.cpu().numpy().astype(int) - 127), 32, axis=1)[:, :H]
        # half an E4M3 step of the value: 2^-4 of it, or 2^-10 of the scale below the normal range
        assert np.all(np.abs(back - rn) <= np.maximum(np.abs(rn) / 16, step / 1024) + 2 * en), "kept rows"
        rc, rs = bl.act8(rn)
        assert (rs == scales.cpu().numpy()).mean() >= 0.99 and (rc == codes.cpu().numpy()).mean() >= 0.98

    # ---- backward ----
    dyt = wide(rows, H, H + pin, t, g, 0.3)
    dres = wide(rows, H, H + pin, t, g, 0.3) if residual else None
    dxb, dx = out_like(rows, H, H + pout, t)
    dgamma, dbeta = torch.empty(H, dtype=wt, device="cuda"), torch.empty(H, dtype=wt, device="cuda")
    ws = torch.full((B.moe_layernorm_workspace_size(n),), 255, dtype=torch.uint8, device="cuda")
    kept = None
    if not act8:
        kept = x
        if residual:                             # what was normalised, at the input pitch
            kept = torch.zeros(rows, H + pin, dtype=t, device="cuda")[:, :H]
            kept.copy_(h)
    B.moe_layernorm_bwd(n, dyt, kept, mean, rstd, codes, scales, gamma, dres, dx, dgamma, dbeta, ws)
    torch.cuda.synchronize()
    rstd64, dy64, gm = f64(rstd), f64(dyt), f64(gamma)
    if act8:
        n64, en = bl.act8_decode(codes.cpu().numpy(), scales.cpu().numpy()), 0.0
    else:
        n64 = (f64(kept) - f64(mean)[:, None]) * rstd64[:, None]
        en = 4 * EPS32 * (np.abs(f64(kept)) + np.abs(f64(mean))[:, None]) * rstd64[:, None]
    rdx, rdg, rdb = bl.layernorm_backward(dy64, n64, rstd64, gm, f64(dres) if residual else None)
    d = np.abs(dy64 * gm)
    an = np.abs(n64)
    e1 = 64 * EPS32 * d.mean(1, keepdims=True)
    e2 = 64 * EPS32 * (d * an).mean(1, keepdims=True) + (d * en).mean(1, keepdims=True)
    m2 = np.abs((dy64 * gm * n64).mean(1, keepdims=True))
    terms = d + d.mean(1, keepdims=True) + an * m2
    slack = rstd64[:, None] * (8 * EPS32 * terms + e1 + an * e2 + en * m2)
    if residual:
        slack = slack + 2 * EPS32 * np.abs(f64(dres))
    assert_within(dx, rdx, slack, "dx")
    assert_within(dgamma, rdg, 512 * EPS32 * (np.abs(dy64) * an).sum(0) + (np.abs(dy64) * en).sum(0), "dgamma")
    assert_within(dbeta, rdb, 512 * EPS32 * np.abs(dy64).sum(0), "dbeta")
    if pout:
        assert bool((dxb[:, H:] == 77.0).all()), "columns past the row were written"
    again_g, again_b = torch.empty_like(dgamma), torch.empty_like(dbeta)
    B.moe_layernorm_bwd(n, dyt, kept, mean, rstd, codes, scales, gamma, dres, dx, again_g, again_b, ws)
    assert torch.equal(again_g, dgamma) and torch.equal(again_b, dbeta), "not reproducible"


def test_gradient_against_differences():
    """The backward pass against central differences of the forward pass itself, in float32: with a
    step of 2^-7 and values of order one the differences are good to about 1e-3 (their rounding,
    2^-24 * 40 / 2^-6, and the third derivative, 2^-14, both stay below)."""
    rows, H = 4, 40
    g = torch.Generator(device="cuda").manual_seed(5)
    n = B.norm(rows, H, x_f32=True, w_f32=True, eps=0.1)
    x, dy = (torch.randn(rows, H, generator=g, device="cuda") for _ in range(2))
    gamma, beta = torch.rand(H, generator=g, device="cuda") + 0.5, torch.zeros(H, device="cuda")
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")

    def loss(v):
        y = torch.empty_like(v)
        B.moe_layernorm_fwd(n, v, None, gamma, beta, None, y, mean, rstd)
        return (y.double() * dy.double()).sum(1)             # rows do not mix

    step = 2.0 ** -7
    diff = torch.empty_like(x)
    for c in range(H):
        a, b = x.clone(), x.clone()
        a[:, c] += step
        b[:, c] -= step
        diff[:, c] = ((loss(a) - loss(b)) / (2 * step)).float()
    loss(x)
    dx, dgamma = torch.empty_like(x), torch.empty_like(gamma)
    ws = torch.zeros(B.moe_layernorm_workspace_size(n), dtype=torch.uint8, device="cuda")
    B.moe_layernorm_bwd(n, dy, x, mean, rstd, None, None, gamma, None, dx, dgamma, None, ws)
    assert float((dx - diff).abs().max()) <= 4e-3


def test_no_rows_and_constant_rows():
    H = 48
    n = B.norm(0, H)
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    dgamma, dbeta = torch.full_like(gamma, 9.0), torch.full_like(gamma, 9.0)
    e = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(B.moe_layernorm_workspace_size(n), dtype=torch.uint8, device="cuda")
    B.moe_layernorm_fwd(n, e, None, gamma, None, None, e, None, None)
    B.moe_layernorm_bwd(n, e, None, None, torch.empty(0, device="cuda"), None, None, gamma, None, e, dgamma, dbeta, ws)
    assert not bool(dgamma.any()) and not bool(dbeta.any())
    # a constant row: n = 0, y = beta; a row with a NaN stays alone with it
    n = B.norm(3, H)
    x = torch.full((3, H), 3.5, dtype=torch.bfloat16, device="cuda")
    x[1, 7] = float("nan")
    beta = torch.arange(H, dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(x)
    codes = torch.empty(3, H, dtype=torch.uint8, device="cuda")
    scales = torch.empty(3, 2, dtype=torch.uint8, device="cuda")
    B.moe_layernorm_fwd(n, x, None, gamma, beta, None, y, None, None, codes, scales)
    assert torch.equal(y[0], beta) and torch.equal(y[2], beta) and bool(y[1].isnan().all())
    assert not bool(codes[0].any()) and bool((scales[1] == 255).all()) and bool((codes[1] == 0x7F).all())


def test_in_place_sum_and_gradient():
    rows, H = 50, 264
    g = torch.Generator(device="cuda").manual_seed(6)
    mk = lambda: torch.randn(rows, H, generator=g, device="cuda").bfloat16()  # noqa: E731
    x, res, dy, dres = mk(), mk(), mk(), mk()
    gamma, beta = torch.ones(H, device="cuda").bfloat16(), torch.zeros(H, device="cuda").bfloat16()
    n = B.norm(rows, H)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    h, y, y2, h2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x), x.clone()
    B.moe_layernorm_fwd(n, x, res, gamma, beta, h, y, mean, rstd)
    B.moe_layernorm_fwd(n, h2, res, gamma, beta, h2, y2, mean, rstd)
    assert torch.equal(h, h2) and torch.equal(y, y2)
    dx, dg = torch.empty_like(x), torch.empty_like(gamma)
    ws = torch.zeros(B.moe_layernorm_workspace_size(n), dtype=torch.uint8, device="cuda")
    B.moe_layernorm_bwd(n, dy, h, mean, rstd, None, None, gamma, dres, dx, dg, None, ws)
    for target in ("dy", "dres"):
        a, b = dy.clone(), dres.clone()
        B.moe_layernorm_bwd(n, a, h, mean, rstd, None, None, gamma, b, a if target == "dy" else b, dg, None, ws)
        assert torch.equal(a if target == "dy" else b, dx), target


def test_on_a_side_stream():
    rows, H = 64, 512
    n = B.norm(rows, H)
    x = torch.randn(rows, H, device="cuda").bfloat16()
    gamma = torch.ones(H, device="cuda").bfloat16()
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    B.moe_layernorm_fwd(n, x, None, gamma, None, None, y, None, None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    B.moe_layernorm_fwd(n, x, None, gamma, None, None, y2, None, None, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, y2)
