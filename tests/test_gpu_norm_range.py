"""Layer norm of finite rows whose sums or squares leave float32's range, against float64.

The norm does not change when a row is multiplied by a power of two (eps aside), so the bounds are those of
ordinary rows: float32 sums with fewer than 64 additions behind any term, the centred value's and the
mean's own roundings, one rounding to the output's type.  Below the normal numbers a mean is a multiple of
2^-149, so a centred value may be off by that much besides.
"""
import numpy as np
import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build
from oracle import block as bl
from rowcheck import EPS32, assert_within, f64

pytestmark = pytest.mark.gpu
F32_MAX = float(np.finfo(np.float32).max)
SHAPES = [(33, True), (40, False), (257, False), (512, True), (2048, False), (4097, True), (16384, False), (16383, True),
          (16384, True)]                              # H, float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def rows_of(kinds, H, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda: torch.randn(H, generator=g, device="cuda", dtype=torch.float64)  # noqa: E731
    sign = torch.where(torch.rand(H, generator=g, device="cuda") < 0.5, -1.0, 1.0).double()
    one_against_all = torch.full((H,), -3.0e38, device="cuda", dtype=torch.float64)
    one_against_all[H // 2] = 3.3e38
    make = {"ordinary": lambda: r(), "squares": lambda: r() * 1e20 + 3e19, "sum": lambda: r().clamp(-8, 8) * 2e37,
            "mean": lambda: r().clamp(-8, 8) * 1e36 + 2.5e38, "both ends": lambda: sign * 3.3e38,
            "one against all": lambda: one_against_all, "constant": lambda: torch.full((H,), 2.0 ** 120, device="cuda").double(),
            "small": lambda: r() * 1e-22, "smaller": lambda: r() * 1e-36 + 1e-36, "subnormal": lambda: r() * 1e-40}
    return torch.stack([make[k]() for k in kinds]).to(dtype)


def forward_and_backward(kinds, H, f32, residual, eps):
    dtype = torch.float32 if f32 else torch.bfloat16
    R = len(kinds)
    g = torch.Generator(device="cuda").manual_seed(H)
    n = B.norm(R, H, x_f32=f32, w_f32=f32, eps=eps)
    x = rows_of(kinds, H, dtype, H)
    res = (x * 0.25).flip(1) if residual else None
    if residual:
        x = (x * 0.5).contiguous()
    gamma = (torch.rand(H, generator=g, device="cuda") + 0.5).to(dtype)
    beta = torch.randn(H, generator=g, device="cuda").to(dtype)
    h, y = torch.empty_like(x) if residual else None, torch.empty_like(x)
    mean, rstd = torch.empty(R, device="cuda"), torch.empty(R, device="cuda")
    codes = torch.zeros(R, H, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(R, (H + 31) // 32, dtype=torch.uint8, device="cuda")
    B.moe_layernorm_fwd(n, x, res, gamma, beta, h, y, mean, rstd, codes, scales)
    x64 = f64(x) + (f64(res) if residual else 0.0)
    ry, rn, rmean, rrstd = bl.layernorm(x64, f64(gamma), f64(beta), eps)
    cen = (np.abs(x64) + np.abs(x64).mean(1, keepdims=True)) * rrstd[:, None]
    rel = 64 * EPS32 * (1 + 2 * (np.abs(rn) * cen).mean(1, keepdims=True))
    en = 64 * EPS32 * cen + np.abs(rn) * rel + 2.0 ** -149 * np.where(np.isfinite(rrstd), rrstd, 0.0)[:, None]
    assert np.all(np.isfinite(ry))
    assert_within(y, ry, en * np.abs(f64(gamma)) + 4 * EPS32 * np.abs(f64(beta)), "y")
    assert_within(mean, rmean, 64 * EPS32 * np.abs(x64).mean(1), "mean")
    seen = np.where(rrstd > F32_MAX, np.inf, rrstd)               # past float32: Inf
    assert_within(rstd, seen, np.where(np.isfinite(seen), rrstd * (rel[:, 0] + 2.0 ** -148 * rrstd), 0.0), "rstd")
    back = bl.act8_decode(codes.cpu().numpy(), scales.cpu().numpy())
    step = np.repeat(np.ldexp(1.0, scales.cpu().numpy().astype(int) - 127), 32, axis=1)[:, :H]
    assert np.all(np.abs(back - rn) <= np.maximum(np.abs(rn) / 16, step / 1024) + 2 * en), "kept rows"
    if residual:
        assert_within(h, x64, EPS32 * np.abs(x64), "h")
    for i, k in enumerate(kinds):
        if k == "constant":
            assert torch.equal(y[i], beta), "a constant row is beta"

    dy = torch.randn(R, H, generator=g, device="cuda").to(dtype)
    dx, dgamma, dbeta = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
    ws = torch.empty(B.moe_layernorm_workspace_size(n), dtype=torch.uint8, device="cuda")
    kept = h if residual else x
    B.moe_layernorm_bwd(n, dy, kept, mean, rstd, None, None, gamma, None, dx, dgamma, dbeta, ws)
    rs = f64(rstd)
    use = np.isfinite(rs)                                         # a gradient past float32 has no bound
    n64 = np.where(use[:, None], (f64(kept) - f64(mean)[:, None]) * np.where(use, rs, 0.0)[:, None], 0.0)
    rdx, rdg, _ = bl.layernorm_backward(f64(dy), n64, np.where(use, rs, 0.0), f64(gamma))
    # (the second term: x or x - mean below the normal numbers, halved or not)
    e = 4 * EPS32 * (np.abs(f64(kept)) + np.abs(f64(mean))[:, None]) * np.where(use, rs, 0.0)[:, None]
    d, an = np.abs(f64(dy) * f64(gamma)), np.abs(n64)
    e2 = 64 * EPS32 * (d * an).mean(1, keepdims=True) + (d * e).mean(1, keepdims=True)
    m2 = np.abs((f64(dy) * f64(gamma) * n64).mean(1, keepdims=True))
    terms = d + d.mean(1, keepdims=True) + an * m2
    slack = np.where(use, rs, 0.0)[:, None] * (8 * EPS32 * terms + 64 * EPS32 * d.mean(1, keepdims=True) + an * e2 + e * m2)
    assert_within(dx[use], rdx[use], slack[use], "dx")
    if use.all():
        assert_within(dgamma, rdg, 512 * EPS32 * (np.abs(f64(dy)) * an).sum(0) + (np.abs(f64(dy)) * e).sum(0), "dgamma")


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("H,f32", SHAPES)
def test_large_rows(H, f32, residual):
    """Rows beside them are ordinary and stay so."""
    kinds = ["ordinary", "squares", "sum", "ordinary", "mean", "both ends", "one against all", "constant", "ordinary"] * 3
    forward_and_backward(kinds, H, f32, residual, 1e-5)


@pytest.mark.parametrize("H,f32", SHAPES)
def test_small_rows_without_eps(H, f32):
    forward_and_backward(["ordinary", "small", "smaller", "ordinary", "subnormal", "squares"] * 3, H, f32, False, 0.0)


def test_rows_that_are_not_finite_stay_alone():
    H = 264
    x = torch.randn(4, H, device="cuda")
    x[1, 3], x[2, 5] = float("inf"), float("nan")
    gamma = torch.ones(H, device="cuda")
    n = B.norm(4, H, x_f32=True, w_f32=True)
    y, mean = torch.empty_like(x), torch.empty(4, device="cuda")
    B.moe_layernorm_fwd(n, x, None, gamma, None, None, y, mean, None)
    assert bool(y[1:3].isnan().all()) and bool(y[[0, 3]].isfinite().all())
    assert float(mean[1]) == float("inf") and bool(mean[2].isnan())


@pytest.mark.parametrize("H,f32", [(2048, False), (33, False), (257, True), (4096, True)])
def test_large_rows_with_the_sum_in_place(H, f32):
    """h in the place of x: float32 stores the sum as it is; in bf16 a row past float32's range is normalised
    as stored, the others from the unrounded sum as ever."""
    dtype = torch.float32 if f32 else torch.bfloat16
    kinds = ["ordinary", "squares", "both ends", "ordinary"] * 4
    x = (rows_of(kinds, H, dtype, H) * 0.5).contiguous()
    res = (x * 0.37).flip(1).contiguous()
    R, ones, zeros = len(kinds), torch.ones(H, dtype=dtype, device="cuda"), torch.zeros(H, dtype=dtype, device="cuda")
    n = B.norm(R, H, x_f32=f32, w_f32=f32)
    y, apart, h = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    B.moe_layernorm_fwd(n, x, res, ones, zeros, h, apart, None, None)
    h2 = x.clone()
    B.moe_layernorm_fwd(n, h2, res, ones, zeros, h2, y, None, None)
    assert torch.equal(h, h2)
    large = torch.tensor([k != "ordinary" for k in kinds], device="cuda")
    assert torch.equal(y[~large], apart[~large])
    if f32:
        assert torch.equal(y, apart)
    x64 = f64(h)
    _, rn, _, rrstd = bl.layernorm(x64, f64(ones), f64(zeros), 1e-5)
    cen = (np.abs(x64) + np.abs(x64).mean(1, keepdims=True)) * rrstd[:, None]
    rel = 64 * EPS32 * (1 + 2 * (np.abs(rn) * cen).mean(1, keepdims=True))
    m = large.cpu().numpy()
    assert_within(y[large], rn[m], (64 * EPS32 * cen + np.abs(rn) * rel)[m], "y")
