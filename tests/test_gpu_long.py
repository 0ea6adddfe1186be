"""Tensors of more than 2^31 elements: the last rows come out as a call on them alone gives them.

A row's result depends on its own values and its length only (norm: threads per row follow from the
length; activation and act8: elementwise apart from dprob), so these are equal bit for bit.  The
linear layers are checked on small whole numbers, whose sums are exact.
"""
import numpy as np
import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build
from oracle import block as bl
from rowcheck import f64

pytestmark = pytest.mark.gpu
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
LAST = 5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    yield
    torch.cuda.empty_cache()


def long_and_last(rows, cols, seed):
    """Zeros with LAST random rows at the end, and those rows by themselves."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    t[-LAST:] = torch.randn(LAST, cols, generator=g, device="cuda").bfloat16()
    return t, t[-LAST:].clone()


@pytest.mark.parametrize("H", [2048, 2047])
def test_layernorm(H):
    rows = 2 ** 31 // H + 1000
    gamma, beta = torch.rand(H, device="cuda").bfloat16(), torch.rand(H, device="cuda").bfloat16()

    def go(x, dy):
        r = x.shape[0]
        n = B.norm(r, H)
        y, dx = torch.empty_like(x), torch.empty_like(x)
        rstd = torch.empty(r, dtype=F32, device="cuda")
        codes = torch.empty(r, H, dtype=U8, device="cuda")
        scales = torch.empty(r, (H + 31) // 32, dtype=U8, device="cuda")
        ws = torch.empty(B.moe_layernorm_workspace_size(n), dtype=U8, device="cuda")
        dg, db = torch.empty_like(gamma), torch.empty_like(beta)
        B.moe_layernorm_fwd(n, x, None, gamma, beta, None, y, None, rstd, codes, scales)
        B.moe_layernorm_bwd(n, dy, None, None, rstd, codes, scales, gamma, None, dx, dg, db, ws)
        return [t[-LAST:].clone() for t in (y, rstd, codes, scales, dx)]

    x, x_last = long_and_last(rows, H, 1)
    dy, dy_last = long_and_last(rows, H, 2)
    for got, want in zip(go(x, dy), go(x_last, dy_last)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("cols", [2048, 2047])
def test_act8(cols):
    rows = 2 ** 31 // cols + 1000

    def go(src):
        codes = torch.empty(src.shape, dtype=U8, device="cuda")
        scales = torch.empty(src.shape[0], (cols + 31) // 32, dtype=U8, device="cuda")
        back = torch.empty_like(src)
        B.moe_act8_pack(src, codes, scales)
        B.moe_act8_unpack(codes, scales, None, None, back)
        return [t[-LAST:].clone() for t in (codes, scales, back)]

    src, last = long_and_last(rows, cols, 3)
    for got, want in zip(go(src), go(last)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("I", [1024, 1023])
def test_swiglu(I):
    rows = 2 ** 31 // (2 * I) + 1000

    def go(gu, da):
        r = gu.shape[0]
        a, dgu = torch.empty(r, I, dtype=BF16, device="cuda"), torch.empty_like(gu)
        codes = torch.empty(r, 2 * I, dtype=U8, device="cuda")
        scales = torch.empty(r, 2 * ((I + 31) // 32), dtype=U8, device="cuda")
        B.moe_swiglu_fwd(gu, None, a, codes, scales)
        B.moe_swiglu_bwd(None, codes, scales, None, da, dgu)
        return [t[-LAST:].clone() for t in (a, codes, scales, dgu)]

    gu, gu_last = long_and_last(rows, 2 * I, 4)
    da, da_last = long_and_last(rows, I, 5)
    for got, want in zip(go(gu, da), go(gu_last, da_last)):
        assert torch.equal(got, want)


def test_grouped_linear():
    K, N, split = 64, 3200, [2 ** 31 // 3200 + 1000, 13]
    rows = sum(split)
    g = torch.Generator(device="cuda").manual_seed(6)
    x, dy = (torch.zeros(rows, c, dtype=BF16, device="cuda") for c in (K, N))
    tern = lambda *s: torch.randint(-1, 2, s, generator=g, device="cuda").bfloat16()  # noqa: E731
    x[-13:] = tern(13, K)
    dy[-13:] = tern(13, N) * (torch.rand(13, N, generator=g, device="cuda") < 0.05)   # sums below 256
    w = tern(2, N, K)
    ss = torch.tensor(split, dtype=torch.int32, device="cuda")
    d = B.grouped(rows, K, N, 2)
    ws = torch.zeros(B.moe_grouped_linear_workspace_size(d), dtype=U8, device="cuda")
    y, dx, dw = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(w)
    B.moe_grouped_linear_fwd(d, x, ss, w, y, ws)
    B.moe_grouped_linear_dgrad(d, dy, ss, w, dx, ws)
    B.moe_grouped_linear_wgrad(d, x, dy, ss, dw, ws)
    assert B.moe_get_device_error(ws) == (0, 0)
    x64, dy64, w64 = f64(x[-13:]), f64(dy[-13:]), f64(w)
    assert np.array_equal(f64(y[-13:]), bl.grouped_linear(x64, w64, [0, 13]))
    assert np.array_equal(f64(dx[-13:]), bl.grouped_linear_dgrad(dy64, w64, [0, 13]))
    assert np.array_equal(f64(dw), bl.grouped_linear_wgrad(x64, dy64, [0, 13]))
    assert not bool(y[:-13].any()) and not bool(dx[:-13].any())
