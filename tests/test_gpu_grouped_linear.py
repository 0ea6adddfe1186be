"""Grouped linear layers on dense ragged rows: forward, dgrad, wgrad against float64.

Two kinds of check.  Small whole numbers: every product and partial sum is exact in float32 and the
result (below 256) exact in bf16, so the outputs must be equal.  Normal values: one rounding to
bf16 plus float32 accumulation, at most C/8 + 16 additions of relative error 2^-23 behind any term
of a sum over C (an MMA step adds 16 terms at once).
"""
import numpy as np
import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build
from oracle import block as bl
from rowcheck import assert_within, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def tensors(split, K, N, rows, seed, whole, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def mk(r, c, lim):
        t = torch.full((r, c + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        t[:, :c] = (torch.randint(-lim, lim + 1, (r, c), generator=g, device="cuda").float() if whole
                    else torch.randn(r, c, generator=g, device="cuda")).bfloat16()
        return t[:, :c]

    x, dy = mk(rows, K, 1), mk(rows, N, 1)
    w = mk(len(split) * N, K + 0, 1).contiguous().view(len(split), N, K)
    if whole:
        # thin out, so that sums stay below 256
        keep = lambda t, c: t.mul_((torch.rand(t.shape, generator=g, device="cuda") < min(1.0, 200.0 / c)).to(t.dtype))  # noqa: E731
        keep(w, max(K, N))
        keep(x, max(split) if len(split) else 1)
    return x, dy, w, torch.tensor(split, dtype=torch.int32, device="cuda")


def run(split, K, N, rows=None, seed=0, whole=True, pad=0):
    rows = sum(split) if rows is None else rows
    x, dy, w, ss = tensors(split, K, N, rows, seed, whole, pad)
    d = B.grouped(rows, K, N, len(split))
    ws = torch.zeros(B.moe_grouped_linear_workspace_size(d), dtype=torch.uint8, device="cuda")
    mk = lambda c: torch.full((rows, c + pad), 77.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    yb, dxb = mk(N), mk(K)
    y, dx = yb[:, :N], dxb[:, :K]
    dw = torch.full((len(split), N, K), 77.0, dtype=torch.bfloat16, device="cuda")
    B.moe_grouped_linear_fwd(d, x, ss, w, y, ws)
    B.moe_grouped_linear_dgrad(d, dy, ss, w, dx, ws)
    B.moe_grouped_linear_wgrad(d, x, dy, ss, dw, ws)
    torch.cuda.synchronize()
    assert B.moe_get_device_error(ws) == (0, 0)
    used = sum(split)
    for full, c in ((yb, N), (dxb, K)):
        assert bool((full[used:] == 77.0).all()), "rows past the sum were written"
        assert bool((full[:, c:] == 77.0).all()), "columns past the row were written"
    return x, dy, w, y, dx, dw, used


def check(split, K, N, **kw):
    x, dy, w, y, dx, dw, used = run(split, K, N, **kw)
    x64, dy64, w64 = f64(x), f64(dy), f64(w)
    refs = (bl.grouped_linear(x64, w64, split)[:used], bl.grouped_linear_dgrad(dy64, w64, split)[:used],
            bl.grouped_linear_wgrad(x64, dy64, split))
    if kw.get("whole", True):
        for name, got, ref in zip(("y", "dx", "dw"), (y[:used], dx[:used], dw), refs):
            assert np.abs(ref).max(initial=0) <= 256, "the inputs of this check are too large to be exact"
            assert np.array_equal(f64(got), ref), name
        return
    ax, ady, aw = np.abs(x64), np.abs(dy64), np.abs(w64)
    err = lambda C: (C / 8 + 16) * 2.0 ** -23  # noqa: E731
    assert_within(y[:used], refs[0], err(K) * bl.grouped_linear(ax, aw, split)[:used], "y")
    assert_within(dx[:used], refs[1], err(N) * bl.grouped_linear_dgrad(ady, aw, split)[:used], "dx")
    assert_within(dw, refs[2], err(max(split)) * bl.grouped_linear_wgrad(ax, ady, split), "dw")


@pytest.mark.parametrize("split,K,N", [
    ([1], 8, 8), ([0, 1], 64, 64), ([3, 0, 2], 72, 40), ([16], 64, 128), ([17, 15], 128, 256),
    ([31, 33, 1, 0, 64], 136, 200), ([128, 129, 127], 256, 264), ([255, 257, 256], 192, 512),
    ([0, 0, 0, 700], 200, 136), ([300, 5, 0, 513], 520, 328), ([1] * 40, 320, 384),
    ([0] * 200 + [3] * 56, 64, 72),
])
def test_whole_numbers(split, K, N):
    check(split, K, N, seed=len(split) + K)


@pytest.mark.parametrize("r", [1, 15, 16, 17, 47, 48, 49, 63, 64, 65, 79, 127, 128, 129, 191, 192, 193])
def test_every_way_an_expert_can_end(r):
    """The contraction of the weight gradient ends inside a step of 64, on a group of 16, in either
    half of a stage; the rows behind it belong to the next expert."""
    check([r, 70, r, 1], 72, 136, seed=r)


@pytest.mark.parametrize("split,K,N", [([5, 0, 130, 300], 1024, 2816), ([700, 68], 2048, 1408), ([1, 2], 4096, 1024)])
def test_normal_values(split, K, N):
    check(split, K, N, whole=False, seed=K)


def test_many_tiles_per_pair():
    """More tiles than CTA pairs, tail stages of several tiles in flight at once."""
    check([33, 1, 70, 5, 129, 18, 0, 3, 250, 45, 7, 66], 1032, 1544, seed=3)


@pytest.mark.parametrize("split,K,N", [([5, 0, 3], 2056, 264), ([1], 8192, 8), ([2, 1], 264, 4104), ([64], 1000, 1000),
                                       ([1, 0, 0, 1], 520, 520), ([30, 2] * 16, 328, 1040)])
def test_tiles_cut_along_the_contraction(split, K, N):
    """Few rows: the tiles of the last round are cut into equal pieces along the contraction.  The second
    call on the same workspace finds the arrival counts as the first did."""
    x, dy, w, ss = tensors(split, K, N, sum(split), K, True)
    d = B.grouped(sum(split), K, N, len(split))
    ws = torch.zeros(B.moe_grouped_linear_workspace_size(d), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        y = torch.full((sum(split), N), 77.0, dtype=torch.bfloat16, device="cuda")
        dx = torch.full((sum(split), K), 77.0, dtype=torch.bfloat16, device="cuda")
        B.moe_grouped_linear_fwd(d, x, ss, w, y, ws)
        B.moe_grouped_linear_dgrad(d, dy, ss, w, dx, ws)
        assert np.array_equal(f64(y), bl.grouped_linear(f64(x), f64(w), split))
        assert np.array_equal(f64(dx), bl.grouped_linear_dgrad(f64(dy), f64(w), split))


def test_rows_past_the_sum_and_pitches():
    check([40, 0, 9], 88, 104, rows=300, seed=4, pad=24)


def test_one_row_does_not_reach_another():
    """NaN and Inf in a row stay in that row's y and dx and in its expert's dw, also where the
    tiles load the neighbours' rows."""
    split, K, N = [21, 45, 30], 136, 72
    x, dy, w, ss = tensors(split, K, N, 100, 9, True)
    d = B.grouped(100, K, N, 3)
    ws = torch.zeros(B.moe_grouped_linear_workspace_size(d), dtype=torch.uint8, device="cuda")

    def go():
        y, dx = torch.zeros(100, N, device="cuda").bfloat16(), torch.zeros(100, K, device="cuda").bfloat16()
        dw = torch.empty(3, N, K, device="cuda").bfloat16()
        B.moe_grouped_linear_fwd(d, x, ss, w, y, ws)
        B.moe_grouped_linear_dgrad(d, dy, ss, w, dx, ws)
        B.moe_grouped_linear_wgrad(d, x, dy, ss, dw, ws)
        return y, dx, dw

    clean = go()
    x[22], dy[22] = float("nan"), float("inf")               # a row of expert 1
    x[97:], dy[97:] = float("nan"), float("nan")             # rows of no expert
    y, dx, dw = go()
    others = [i for i in range(100) if i != 22]
    assert torch.equal(y[others], clean[0][others]) and torch.equal(dx[others], clean[1][others])
    assert bool(y[22].isnan().all()) and not bool(dx[22].isfinite().all())
    assert torch.equal(dw[0], clean[2][0]) and torch.equal(dw[2], clean[2][2]) and bool(dw[1].isnan().all())


@pytest.mark.parametrize("split", [[5, -1, 4], [5, 60, 4], [2 ** 30, 2 ** 30, 2 ** 30]])
def test_inconsistent_sizes_are_recorded_and_write_nothing(split):
    x, dy, w, _ = tensors([5, 3, 4], 64, 64, 40, 1, True)
    ss = torch.tensor(split, dtype=torch.int32, device="cuda")
    d = B.grouped(40, 64, 64, 3)
    for mode in range(3):
        ws = torch.zeros(B.moe_grouped_linear_workspace_size(d), dtype=torch.uint8, device="cuda")
        out = torch.full((3, 64, 64) if mode == 2 else (40, 64), 77.0, dtype=torch.bfloat16, device="cuda")
        if mode == 0:
            B.moe_grouped_linear_fwd(d, x, ss, w, out, ws)
        elif mode == 1:
            B.moe_grouped_linear_dgrad(d, dy, ss, w, out, ws)
        else:
            B.moe_grouped_linear_wgrad(d, x, dy, ss, out, ws)
        assert B.moe_get_device_error(ws)[0] == 7
        assert bool((out == 77.0).all())


def test_no_rows():
    d = B.grouped(0, 64, 64, 3)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(3, 64, 64, dtype=torch.bfloat16, device="cuda")
    ss = torch.zeros(3, dtype=torch.int32, device="cuda")
    ws = torch.zeros(B.moe_grouped_linear_workspace_size(d), dtype=torch.uint8, device="cuda")
    B.moe_grouped_linear_fwd(d, e, ss, w, e, ws)
    B.moe_grouped_linear_dgrad(d, e, ss, w, e, ws)
    B.moe_grouped_linear_wgrad(d, e, e, ss, w, ws)
    assert not bool(w.any())


@pytest.mark.parametrize("rows,K,N", [(1, 64, 64), (40, 1032, 520), (3000, 256, 136)])
def test_rows_but_no_expert_has_any(rows, K, N):
    x, dy, w, _ = tensors([rows], K, N, rows, 2, True)
    w = w.expand(3, N, K).contiguous()
    ss = torch.zeros(3, dtype=torch.int32, device="cuda")
    d = B.grouped(rows, K, N, 3)
    ws = torch.zeros(B.moe_grouped_linear_workspace_size(d), dtype=torch.uint8, device="cuda")
    y, dx, dw = (torch.full(s, 77.0, dtype=torch.bfloat16, device="cuda") for s in ((rows, N), (rows, K), (3, N, K)))
    B.moe_grouped_linear_fwd(d, x, ss, w, y, ws)
    B.moe_grouped_linear_dgrad(d, dy, ss, w, dx, ws)
    B.moe_grouped_linear_wgrad(d, x, dy, ss, dw, ws)
    assert B.moe_get_device_error(ws) == (0, 0)
    assert bool((y == 77.0).all()) and bool((dx == 77.0).all()) and not bool(dw.any())


def test_reproducible():
    a, b = run([100, 33, 250], 264, 520, whole=False), run([100, 33, 250], 264, 520, whole=False)
    for i in (3, 4, 5):
        assert torch.equal(a[i], b[i])
