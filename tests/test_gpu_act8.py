"""8-bit checkpoints and the gated activation on the GPU.

act8 codes and scales of bf16 and f32 input are compared bit for bit with the oracle.  The
activation's bounds: one rounding to the output's type plus float32 arithmetic, where the
exponential's error is 2 + 1.2 |g| units in the last place and every other step a unit or two.
"""
import numpy as np
import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build
from oracle import block as bl
from rowcheck import EPS32, assert_within, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def values(rows, cols, g, dtype):
    """Rows of very different size, with zeros, an all-zero row, subnormals, and values on the
    rule's boundaries (1.75 * 2^k and the ties between two codes)."""
    v = torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(4 * torch.randn(rows, 1, generator=g, device="cuda"))
    v[torch.rand(rows, cols, generator=g, device="cuda") < 0.05] = 0.0
    k = torch.randint(-6, 9, (rows, cols), generator=g, device="cuda").float()
    tie = (1.0 + torch.randint(0, 16, (rows, cols), generator=g, device="cuda").float() / 16) * torch.exp2(k)
    v[1::3] = tie[1::3]
    if rows > 2:
        v[2] = 0.0
    if rows > 5:
        v[5] = v[5] * 1e-38
    return v.to(dtype)


def new_act8(rows, cols):
    return (torch.full((rows, cols), 0x55, dtype=torch.uint8, device="cuda"),
            torch.full((rows, (cols + 31) // 32), 0x55, dtype=torch.uint8, device="cuda"))


SIZES = [(1, 1), (2, 8), (6, 31), (7, 32), (3, 33), (40, 1000), (517, 1003), (9, 5632), (1300, 72)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_pack_and_unpack(rows, cols, dtype):
    g = torch.Generator(device="cuda").manual_seed(rows + cols)
    v = values(rows, cols, g, dtype)
    codes, scales = new_act8(rows, cols)
    B.moe_act8_pack(v, codes, scales)
    rc, rs = bl.act8(f64(v))
    assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)
    back = bl.act8_decode(rc, rs)
    for out in (torch.float32, torch.bfloat16):
        d = torch.full((rows, cols + 5), 77.0, dtype=out, device="cuda")
        B.moe_act8_unpack(codes, scales, None, None, d[:, :cols])
        assert bool((d[:, cols:] == 77.0).all())
        want = torch.from_numpy(back).to(torch.float32).to(out)       # exact in float32
        assert torch.equal(d[:, :cols].cpu(), want)


@pytest.mark.parametrize("cols", [64, 65])
@pytest.mark.parametrize("wt", [torch.bfloat16, torch.float32])
def test_unpack_with_weights(cols, wt):
    g = torch.Generator(device="cuda").manual_seed(cols)
    v = torch.randn(20, cols, generator=g, device="cuda")
    codes, scales = new_act8(20, cols)
    B.moe_act8_pack(v, codes, scales)
    gamma = torch.randn(cols, generator=g, device="cuda").to(wt)
    beta = torch.randn(cols, generator=g, device="cuda").to(wt)
    back = bl.act8_decode(codes.cpu().numpy(), scales.cpu().numpy())
    for b in (None, beta):
        d = torch.empty(20, cols, dtype=torch.bfloat16, device="cuda")
        B.moe_act8_unpack(codes, scales, gamma, b, d)
        ref = back * f64(gamma) + (0.0 if b is None else f64(b))
        assert_within(d, ref, 2 * EPS32 * (np.abs(back * f64(gamma)) + np.abs(f64(beta))), "dst")


def test_pack_strided_and_not_finite():
    v = torch.randn(6, 96, device="cuda")
    v[1, 40], v[3, 0], v[4, 95] = float("inf"), float("nan"), float("-inf")
    for cols in (80, 77):
        codes, scales = new_act8(6, cols)
        B.moe_act8_pack(v[:, :cols], codes, scales)
        rc, rs = bl.act8(f64(v[:, :cols]))
        assert np.array_equal(codes.cpu().numpy(), rc) and np.array_equal(scales.cpu().numpy(), rs)
        d = torch.empty(6, cols, device="cuda")
        B.moe_act8_unpack(codes, scales, None, None, d)
        assert np.array_equal(np.isnan(f64(d)), np.isnan(bl.act8_decode(rc, rs)))


def test_no_rows():
    e8, e16 = torch.empty(0, 32, dtype=torch.uint8, device="cuda"), torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    B.moe_act8_pack(e16, e8, e8)
    B.moe_act8_unpack(e8, e8, None, None, e16)
    B.moe_swiglu_fwd(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), None, e16)


CASES = [
    # rows, I, prob, act8, pitches beyond the rows
    (1, 1, True, True, 0), (1, 8, False, True, 0), (3, 31, True, True, 0), (5, 40, True, True, 8),
    (7, 32, True, False, 0), (12, 1408, True, True, 0), (130, 264, True, True, 0), (33, 1001, True, True, 3),
    (33, 1001, False, False, 0), (2600, 96, True, True, 0), (4, 14336, True, True, 0), (40, 2816, True, False, 8),
    # rows enough that a warp takes a row by itself, several steps long
    (9800, 520, True, True, 0),
]


@pytest.mark.parametrize("rows,I,with_prob,act8,pad", CASES)
def test_swiglu(rows, I, with_prob, act8, pad):
    g = torch.Generator(device="cuda").manual_seed(rows * 3 + I)

    def mat(cols, std=1.0, fill=float("nan")):
        t = torch.full((rows, cols + pad), fill, dtype=torch.bfloat16, device="cuda")
        t[:, :cols] = (torch.randn(rows, cols, generator=g, device="cuda") * std).bfloat16()
        return t, t[:, :cols]

    _, gu = mat(2 * I, 3.0)
    if rows > 2:
        gu[2, :I] = torch.linspace(-88, 88, I, device="cuda").bfloat16()        # far ends of the sigmoid
        gu[1, 0] = 0.0
    prob = torch.rand(rows, generator=g, device="cuda") if with_prob else None
    ab, a = mat(I, fill=77.0)
    codes, scales = None, None
    if act8:
        codes = torch.empty(rows, 2 * I, dtype=torch.uint8, device="cuda")
        scales = torch.empty(rows, 2 * ((I + 31) // 32), dtype=torch.uint8, device="cuda")
    B.moe_swiglu_fwd(gu, prob, a, codes, scales)
    torch.cuda.synchronize()
    g64, u64 = f64(gu[:, :I]), f64(gu[:, I:])
    p64 = f64(prob) if with_prob else np.ones(rows)

    def ulps(gg):
        return EPS32 * (16 + 4 * np.abs(gg))

    ra = bl.swiglu(g64, u64, p64)
    # below float32's range the sigmoid is zero: 2^-126 of g * u * p
    under = 2.0 ** -125 * np.abs(g64 * u64)
    assert_within(a, ra, ulps(g64) * np.abs(ra) + under, "a")
    if act8:
        nb = (I + 31) // 32
        for half, ref in ((slice(0, I), g64), (slice(I, 2 * I), u64)):
            rc, rs = bl.act8(ref)
            assert np.array_equal(codes[:, half].cpu().numpy(), rc)
            blk = slice(0, nb) if half.start == 0 else slice(nb, 2 * nb)
            assert np.array_equal(scales[:, blk].cpu().numpy(), rs)
        g64 = bl.act8_decode(codes[:, :I].cpu().numpy(), scales[:, :nb].cpu().numpy())
        u64 = bl.act8_decode(codes[:, I:].cpu().numpy(), scales[:, nb:].cpu().numpy())

    _, da = mat(I, 0.5)
    dgub, dgu = mat(2 * I, fill=77.0)
    a2b, a2 = mat(I, fill=77.0)
    dprob = torch.empty(rows, device="cuda") if with_prob else None
    B.moe_swiglu_bwd(None if act8 else gu, codes, scales, prob, da, dgu, dprob, a2)
    torch.cuda.synchronize()
    da64 = f64(da)
    rdg, rdu, rdp = bl.swiglu_backward(g64, u64, p64, da64)
    s = 1.0 / (1.0 + np.exp(-g64))
    size = np.abs(da64 * p64[:, None])
    under = 2.0 ** -125
    # silu' = s + g s (1 - s): the sum of its terms' magnitudes carries the error
    mag = size * np.abs(u64) * (s + np.abs(g64) * s * (1 - s) + np.abs(g64) * s * EPS32)
    assert_within(dgu[:, :I], rdg, ulps(g64) * mag + under * size * np.abs(u64) * (1 + np.abs(g64)), "dg")
    assert_within(dgu[:, I:], rdu, ulps(g64) * np.abs(rdu) + under * size * np.abs(g64), "du")
    ra = bl.swiglu(g64, u64, p64)
    assert_within(a2, ra, ulps(g64) * np.abs(ra) + under * np.abs(g64 * u64), "a again")
    if with_prob:
        terms = np.abs(da64 * g64 * s * u64)
        # fewer than 64 + I / 256 additions behind any term
        assert_within(dprob, rdp, ((64 + I / 256) * EPS32 + ulps(g64)) .__mul__(terms).sum(1) + 1e-30, "dprob")
    if pad:
        for t, c in ((ab, I), (dgub, 2 * I), (a2b, I)):
            assert bool((t[:, c:] == 77.0).all()), "columns past the row were written"


def test_swiglu_in_place_and_without_extras():
    rows, I = 20, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    gu = torch.randn(rows, 2 * I, generator=g, device="cuda").bfloat16()
    da = torch.randn(rows, I, generator=g, device="cuda").bfloat16()
    prob = torch.rand(rows, generator=g, device="cuda")
    d1, d2, a = torch.empty_like(gu), torch.empty_like(gu), torch.empty_like(da)
    B.moe_swiglu_bwd(gu, None, None, prob, da, d1, None, a)
    both = da.clone()
    B.moe_swiglu_bwd(gu, None, None, prob, both, d2, None, both)          # a takes da's place
    assert torch.equal(d1, d2) and torch.equal(both, a)
    d3 = torch.empty_like(gu)
    B.moe_swiglu_bwd(gu, None, None, prob, da, d3)
    assert torch.equal(d1, d3)


def test_swiglu_gradient_against_differences():
    """dg, du, dp from kept bf16 values against central differences of the float64 formula, whose
    error at this step is below 1e-7; what remains is one rounding to bf16."""
    rows, I = 4, 24
    g = torch.Generator(device="cuda").manual_seed(2)
    gu = torch.randn(rows, 2 * I, generator=g, device="cuda").bfloat16()
    da = torch.randn(rows, I, generator=g, device="cuda").bfloat16()
    prob = torch.rand(rows, generator=g, device="cuda")
    dgu, dprob = torch.empty_like(gu), torch.empty(rows, device="cuda")
    B.moe_swiglu_bwd(gu, None, None, prob, da, dgu, dprob)
    v, p, d = f64(gu), f64(prob), f64(da)
    h = 1e-5
    loss = lambda v, p: (bl.swiglu(v[:, :I], v[:, I:], p) * d)  # noqa: E731
    diff = np.zeros_like(v)
    for c in range(2 * I):
        a, b = v.copy(), v.copy()
        a[:, c] += h
        b[:, c] -= h
        diff[:, c] = ((loss(a, p) - loss(b, p)) / (2 * h)).sum(1)
    assert_within(dgu, diff, 1e-6, "dgu")
    assert_within(dprob, ((loss(v, p + h) - loss(v, p - h)) / (2 * h)).sum(1), 1e-5, "dprob")
