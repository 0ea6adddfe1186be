"""The root-mean-square norm where a row group has several rows and some of them have squares that float32 cannot hold.

Such rows are normalised in a loop behind the kernel's, which goes past the others.  5000 rows are five or nine a
group here, so groups of an even and of an odd number of rows are among them.  Tolerances are those of
test_gpu_rmsnorm.py: e = (H / 64 + 16) 2^-24 for rstd and the product with it, one rounding of the float32 sum x + residual
(relative to the sum, and to its square's root again) more where there is a residual.
"""
import numpy as np
import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build
from oracle import fp8_block as fb
from rowcheck import EPS32, assert_within, f64

pytestmark = pytest.mark.gpu
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
LARGE, SMALL = {BF16: 1e38, F32: 2e38}, {BF16: 1e-30, F32: 1e-30}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def rows(R, H, xt, odd, size, seed):
    """Ordinary rows, those of `odd` of the given size (all of one magnitude to a factor of two)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(R, H, generator=g, device="cuda")
    x[odd] = (torch.rand(int(odd.sum()), H, generator=g, device="cuda") * 0.5 + 0.5) * size
    return x.to(xt)


def picked(R, which):
    i = torch.arange(R, device="cuda")
    return {"every third": i % 3 == 2, "the last": i == R - 1, "all but every third": i % 3 != 0, "the first thousand": i < 1000}[which]


@pytest.mark.parametrize("which", ["every third", "the last", "all but every third", "the first thousand"])
@pytest.mark.parametrize("R,H,xt", [(5000, 2048, BF16), (5000, 2048, F32), (5000, 1001, BF16), (4999, 1001, F32), (5000, 4096, BF16),
                                    (1300, 16384, BF16), (1300, 8200, F32), (9001, 512, BF16), (30000, 136, BF16)])
def test_among_rows_of_the_same_group(R, H, xt, which):
    odd = picked(R, which)
    for size, eps in ((LARGE[xt], 1e-5), (SMALL[xt], 0.0)):
        x = rows(R, H, xt, odd, size, R + H)
        n = B.norm(R, H, x_f32=xt == F32, eps=eps)
        y, rstd = torch.full((R, H), 77.0, dtype=xt, device="cuda"), torch.full((R,), 77.0, device="cuda")
        gamma = torch.ones(H, dtype=BF16, device="cuda")
        B.moe_rmsnorm_fwd(n, x, None, gamma, None, y, rstd)
        ry, _, rr = fb.rmsnorm(f64(x), f64(gamma), float(np.float32(eps)))
        assert_within(y, ry, (H / 64 + 16) * EPS32 * np.abs(ry), "y")
        assert np.all(np.abs(f64(rstd) - rr) <= (H / 64 + 16) * EPS32 * rr + 2.0 ** -149)


@pytest.mark.parametrize("place", ["x", "residual", "neither"])
@pytest.mark.parametrize("R,H,xt", [(5000, 2048, BF16), (5000, 1001, BF16), (5000, 2048, F32), (700, 1001, F32), (9, 264, BF16)])
def test_h_in_the_place_of_x_or_the_residual(R, H, xt, place):
    """h holds the sum there when the second loop comes; a row out of range is then the one that h holds."""
    odd = picked(R, "every third")
    for size, eps in ((LARGE[xt], 1e-5), (SMALL[xt], 0.0)):
        x = rows(R, H, xt, odd, size, R)
        res = rows(R, H, xt, odd, size * 0.25, R + 1)
        x0, res0 = f64(x), f64(res)
        n = B.norm(R, H, x_f32=xt == F32, eps=eps)
        h = {"x": x, "residual": res, "neither": torch.full_like(x, 77.0)}[place]
        y, rstd = torch.full((R, H), 77.0, dtype=xt, device="cuda"), torch.full((R,), 77.0, device="cuda")
        gamma = torch.ones(H, dtype=BF16, device="cuda")
        B.moe_rmsnorm_fwd(n, x, res, gamma, h, y, rstd)
        assert_within(h, x0 + res0, 2 * EPS32 * np.abs(x0 + res0), "h")
        want = x0 + res0
        if place != "neither":
            want = np.where(odd.cpu().numpy()[:, None], f64(h), want)
        ry, _, rr = fb.rmsnorm(want, f64(gamma), float(np.float32(eps)))
        # the float32 sum: 2^-24 of itself where it is a normal number, as here
        assert_within(y, ry, (H / 64 + 16 + 3 + 4) * EPS32 * np.abs(ry), "y")
        assert np.all(np.abs(f64(rstd) - rr) <= (H / 64 + 16 + 2) * EPS32 * rr + 2.0 ** -149)


@pytest.mark.parametrize("R,H", [(5000, 2048), (4999, 1001)])
def test_reproducible(R, H):
    odd = picked(R, "every third")
    x = rows(R, H, BF16, odd, 1e38, 5)
    gamma, n = torch.ones(H, dtype=BF16, device="cuda"), B.norm(R, H)
    got = []
    for _ in range(8):
        y, rstd = torch.zeros(R, H, dtype=BF16, device="cuda"), torch.zeros(R, device="cuda")
        codes, scales = torch.zeros(R, H, dtype=U8, device="cuda"), torch.zeros(-(-H // 128), R, device="cuda")
        B.moe_rmsnorm_fwd(n, x, None, gamma, None, y, rstd, codes, scales)
        got.append((y, rstd, codes, scales))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
