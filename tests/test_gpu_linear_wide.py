"""Grouped linear layers in tiles of up to 512 columns on two accumulators, against exact products.

Such tiles are taken where they make four rounds for every CTA pair.  Whole numbers: every sum is exact in
float32 and, at most 256, in bf16, so the results have to be equal.  Experts end in every part of a tile;
contractions of one to seven steps of 64 let a tile's first accumulator run ahead of the second in full,
in part and not at all.
"""
import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build

pytestmark = pytest.mark.gpu
# rows of experts: none, inside the first half, at its end, inside the second, several tiles
ROWS = [257, 288, 0, 320, 480, 511, 512, 513, 1, 33, 256, 700, 769, 800, 1023, 1024, 300, 449, 497, 385]
CONTRACTIONS = [8, 72, 128, 136, 200, 264, 448]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    yield
    torch.cuda.empty_cache()


def pairs():
    return torch.cuda.get_device_properties(0).multi_processor_count // 2


def ternary(g, *s):
    return torch.randint(-1, 2, s, generator=g, device="cuda").bfloat16()


def setup(split, K, N, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    d = B.grouped(sum(split), K, N, len(split))
    ws = torch.zeros(B.moe_grouped_linear_workspace_size(d), dtype=torch.uint8, device="cuda")
    return g, d, ws, torch.tensor(split, dtype=torch.int32, device="cuda")


def by_expert(split):
    a = 0
    for e, s in enumerate(split):
        yield e, slice(a, a + s)
        a += s


def check(got, want, name):
    assert float(want.abs().max()) <= 256, "the inputs of this check are too large to be exact"
    bad = got.float() != want
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("C", CONTRACTIONS)
@pytest.mark.parametrize("dgrad", [False, True], ids=["forward", "dgrad"])
def test_rows_in_wide_tiles(dgrad, C):
    M, split = 8200, ROWS * 2                    # 33 tiles of 256 features, the last of 8
    R, E = sum(split), len(split)
    assert (M + 255) // 256 * (R // 512) >= 4 * pairs(), "no wide tiles at these sizes"
    K, N = (M, C) if dgrad else (C, M)
    g, d, ws, ss = setup(split, K, N, C)
    rows_in, w = ternary(g, R, C), ternary(g, E, N, K)
    out = torch.full((R, M), 77, dtype=torch.bfloat16, device="cuda")
    (B.moe_grouped_linear_dgrad if dgrad else B.moe_grouped_linear_fwd)(d, rows_in, ss, w, out, ws)
    want = torch.empty(R, M, device="cuda")
    for e, s in by_expert(split):
        want[s] = rows_in[s].float() @ (w[e].float() if dgrad else w[e].float().t())
    check(out, want, "dx" if dgrad else "y")
    assert B.moe_get_device_error(ws) == (0, 0)


@pytest.mark.parametrize("n", [8, 64, 136, 192, 264, 320, 392, 448, 504, 512])
@pytest.mark.parametrize("K", [1544, 1536])
def test_weight_gradient_in_wide_tiles(K, n):
    """n: columns of the last tile.  K and N multiples of 64 or not: two kernels.  Experts whose rows are no
    multiple of 16 have their last step cleared behind them, in up to four blocks of 64 columns."""
    N = 2048 + n
    split = [17, 33, 64, 100, 129, 16, 15, 1, 0, 250, 63, 200, 240, 47]
    R, E = sum(split), len(split)
    assert E * ((N + 511) // 512) * ((K + 255) // 256) >= 4 * pairs(), "no wide tiles at these sizes"
    g, d, ws, ss = setup(split, K, N, n)
    x, dy = ternary(g, R, K), ternary(g, R, N)
    dw = torch.full((E, N, K), 77, dtype=torch.bfloat16, device="cuda")
    B.moe_grouped_linear_wgrad(d, x, dy, ss, dw, ws)
    want = torch.empty(E, N, K, device="cuda")
    for e, s in by_expert(split):
        want[e] = dy[s].float().t() @ x[s].float()
    check(dw, want, "dw")
    assert B.moe_get_device_error(ws) == (0, 0)
