"""Grouped linear layers on 8-bit operands with scales of blocks of 128: forward, dgrad, wgrad against float64.

Two kinds of check.  Codes of -1, 0, 1 and scales that are powers of two: every product and partial sum is
exact in float32, so an output is its exact sum rounded once to bf16.  Codes of normal values and any scales:
one rounding to bf16 plus float32 accumulation, at most C/8 + 16 additions of relative error 2^-23 behind any
term of a sum over C, and four more roundings of 2^-24 behind it (the product of the scales, and the block's
sum times it).
"""
import numpy as np
import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build
from oracle import fp8_block as fb
from rowcheck import assert_within, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def bf16(v):
    return torch.tensor(v).to(torch.bfloat16).to(torch.float64).numpy()


class Case:
    """Random operands of one layer in all four forms, codes and scales."""

    def __init__(self, split, K, N, rows, seed, whole):
        self.split, self.K, self.N, self.rows, self.E = split, K, N, rows, len(split)
        rng = np.random.default_rng(seed)
        cut = lambda n: -(-n // 128)  # noqa: E731
        blocks = B.fp8_blocks(rows, self.E)

        def codes(*shape, dim=-1):
            if whole:
                return rng.choice(np.array([0, 0x38, 0xB8], dtype=np.uint8), shape)
            return fb.encode(rng.normal(size=shape) * 60)

        def scales(*shape):
            if whole:
                return (2.0 ** rng.integers(-2, 3, shape)).astype(np.float32)
            return np.exp(rng.normal(size=shape)).astype(np.float32)

        self.host = {"x": codes(rows, K), "xs": scales(cut(K), rows), "dy": codes(rows, N), "dys": scales(cut(N), rows),
                     "w": codes(self.E, N, K), "ws": scales(self.E, cut(N), cut(K)),
                     "xt": codes(blocks * 128, K), "xts": scales(blocks, cut(K)),
                     "dyt": codes(blocks * 128, N), "dyts": scales(blocks, N)}
        first, used = fb.layout(split)
        for n, f in zip(split, first):                       # rows past an expert's last are zeros
            end = f + -(-n // 128) * 128
            self.host["xt"][f + n: end] = 0
            self.host["dyt"][f + n: end] = 0
        self.first = first
        self.dev = {k: torch.tensor(v, device="cuda") for k, v in self.host.items()}
        self.ss = torch.tensor(split, dtype=torch.int32, device="cuda")
        self.g = B.grouped(rows, K, N, self.E)
        self.ws = torch.zeros(B.moe_grouped_linear_fp8_workspace_size(self.g), dtype=torch.uint8, device="cuda")

    def run(self, pad=0):
        d, g = self.dev, self.g
        mk = lambda c: torch.full((self.rows, c + pad), 77.0, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        yb, dxb = mk(self.N), mk(self.K)
        y, dx = yb[:, : self.N], dxb[:, : self.K]
        dw = torch.full((self.E, self.N, self.K), 77.0, dtype=torch.bfloat16, device="cuda")
        B.moe_grouped_linear_fp8_fwd(g, d["x"], d["xs"], self.ss, d["w"], d["ws"], y, self.ws)
        B.moe_grouped_linear_fp8_dgrad(g, d["dy"], d["dys"], self.ss, d["w"], d["ws"], dx, self.ws)
        B.moe_grouped_linear_fp8_wgrad(g, d["xt"], d["xts"], d["dyt"], d["dyts"], self.ss, dw, self.ws)
        torch.cuda.synchronize()
        assert B.moe_get_device_error(self.ws) == (0, 0)
        used = sum(self.split)
        for full, c in ((yb, self.N), (dxb, self.K)):
            assert bool((full[used:] == 77.0).all()), "rows past the sum were written"
            assert bool((full[:, c:] == 77.0).all()), "columns past the row were written"
        return y[:used], dx[:used], dw

    def exact(self, of=lambda v: v):
        """y, dx, dw in float64, of the operands' values or of `of` them."""
        h = self.host
        used = sum(self.split)
        y, dx, dw = np.zeros((used, self.N)), np.zeros((used, self.K)), np.zeros((self.E, self.N, self.K))
        x, dy = of(fb.rows_back(h["x"], h["xs"])), of(fb.rows_back(h["dy"], h["dys"]))
        xt, dyt = of(fb.tiles_back(h["xt"], h["xts"])), of(fb.tokens_back(h["dyt"], h["dyts"]))
        r0 = 0
        for e, n in enumerate(self.split):
            w, f = of(fb.tiles_back(h["w"][e], h["ws"][e])), self.first[e]
            y[r0: r0 + n], dx[r0: r0 + n] = x[r0: r0 + n] @ w.T, dy[r0: r0 + n] @ w
            dw[e] = dyt[f: f + n].T @ xt[f: f + n]
            r0 += n
        return y, dx, dw


def check_whole(split, K, N, rows=None, seed=0, pad=0):
    c = Case(split, K, N, sum(split) if rows is None else rows, seed, True)
    for name, got, ref in zip(("y", "dx", "dw"), c.run(pad), c.exact()):
        assert np.array_equal(f64(got), bf16(ref)), name


@pytest.mark.parametrize("split,K,N", [
    ([1], 16, 16), ([1], 128, 128), ([0, 1], 64, 64), ([3, 0, 2], 80, 48), ([128], 256, 256), ([16], 64, 128),
    ([17, 15], 128, 272), ([31, 33, 1, 0, 64], 144, 208), ([128, 129, 127], 256, 272), ([255, 257, 256], 192, 512),
    ([0, 0, 0, 700], 208, 144), ([300, 5, 0, 513], 528, 336), ([1] * 40, 320, 384), ([0] * 200 + [3] * 56, 64, 80),
])
def test_whole_numbers(split, K, N):
    check_whole(split, K, N, seed=len(split) + K)


@pytest.mark.parametrize("r", [1, 31, 32, 33, 64, 95, 96, 97, 127, 128, 129, 159, 160, 161, 255, 256, 257])
def test_every_way_an_expert_can_end(r):
    check_whole([r, 70, r, 1], 112, 144, seed=r)


@pytest.mark.parametrize("c", [16, 48, 112, 128, 144, 240, 256, 272, 400])
def test_every_way_a_row_can_end(c):
    check_whole([40, 130], c, 16, seed=c)
    check_whole([40, 130], 16, c, seed=c + 1)


@pytest.mark.parametrize("split,K,N", [([5, 0, 130, 300], 1024, 2816), ([700, 68], 2048, 1408), ([1, 2], 4096, 1024)])
def test_normal_values(split, K, N):
    c = Case(split, K, N, sum(split), K, False)
    err = lambda C: (C / 8 + 20) * 2.0 ** -23  # noqa: E731
    for name, got, ref, size, C in zip(("y", "dx", "dw"), c.run(), c.exact(), c.exact(np.abs), (K, N, max(split))):
        assert_within(got, ref, err(C) * size, name)


def test_many_tiles_per_pair():
    check_whole([33, 1, 70, 5, 129, 18, 0, 3, 250, 45, 7, 66], 1040, 1552, seed=3)
    check_whole([900, 1, 2100], 784, 4624, seed=4)


@pytest.mark.parametrize("split,K,N", [([5, 0, 3], 2064, 272), ([1], 8192, 16), ([2, 1], 272, 4112), ([64], 1008, 1008),
                                       ([1, 0, 0, 1], 528, 528), ([30, 2] * 16, 336, 1040), ([1], 14336, 4096), ([17], 4096, 2048),
                                       ([48, 33, 16], 640, 400), ([0, 65, 0, 130], 1024, 272)])
def test_few_rows(split, K, N):
    """Tiles of 64 rows, cut along the contraction.  The later calls on the same workspace find the arrival counts
    as the first did."""
    c = Case(split, K, N, sum(split), K, True)
    ref = [bf16(v) for v in c.exact()]
    for _ in range(3):
        for name, got, want in zip(("y", "dx", "dw"), c.run(), ref):
            assert np.array_equal(f64(got), want), name


@pytest.mark.parametrize("split,K,N", [([40000], 48, 32), ([9000, 0, 4100, 1, 130], 272, 256), ([30000] + [1] * 40, 64, 144),
                                       ([6000, 6000, 5999], 528, 784), ([4097], 16, 16), ([4096 + 128 * 77, 5], 32, 16), ([3] * 100 + [5000] + [2] * 155, 16, 32), ([20] * 255 + [9000], 48, 16), ([20000, 900], 1040, 2064)])
def test_weight_gradient_of_few_long_tiles(split, K, N):
    """Tiles that are cut along the rows: several experts, ends of every kind, and a workspace used again.  Codes of -1,
    0 and 1: sums of up to 40000 such products, of variance 0.44, stay below 2^24, and scales of one keep them whole."""
    R, E = sum(split), len(split)
    g, nb = B.grouped(R, K, N, E), B.fp8_blocks(R, E)
    ss = torch.tensor(split, dtype=torch.int32, device="cuda")
    ws = torch.zeros(B.moe_grouped_linear_fp8_workspace_size(g), dtype=torch.uint8, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(R)
    pick = torch.tensor([0xB8, 0x00, 0x38], dtype=torch.uint8, device="cuda")
    xt, dyt = (pick[torch.randint(0, 3, (nb * 128, c), generator=gen, device="cuda")] for c in (K, N))
    at, ref = 0, torch.zeros(E, N, K, dtype=torch.float64, device="cuda")
    for e, n in enumerate(split):
        end = at + -(-n // 128) * 128
        dyt[at + n: end] = 0                                 # as the quantizer leaves them
        xt[at + n: end] = 0
        x, dy = (t[at:end].view(torch.float8_e4m3fn).double() for t in (xt, dyt))
        ref[e] = dy.T @ x
        at = end
    one = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    for _ in range(2):
        dw = torch.full((E, N, K), 77.0, dtype=torch.bfloat16, device="cuda")
        B.moe_grouped_linear_fp8_wgrad(g, xt, one(nb, -(-K // 128)), dyt, one(nb, N), ss, dw, ws)
        assert B.moe_get_device_error(ws) == (0, 0)
        assert torch.equal(dw, ref.to(torch.bfloat16))


def test_weight_gradient_of_many_rows_that_no_expert_has():
    """The path that cuts tiles, with nothing to cut: zeros where no expert has rows, nothing at all where the sizes do
    not fit."""
    R, K, N, E = 6000, 32, 48, 3
    g, nb = B.grouped(R, K, N, E), B.fp8_blocks(R, E)
    u8 = lambda *s: torch.full(s, 0x38, dtype=torch.uint8, device="cuda")  # noqa: E731
    one = lambda *s: torch.ones(*s, device="cuda")  # noqa: E731
    for split, want, code in (([0, 0, 0], 0.0, 0), ([6000, 1, 0], 77.0, 7), ([-1, 5000, 0], 77.0, 7)):
        ws = torch.zeros(B.moe_grouped_linear_fp8_workspace_size(g), dtype=torch.uint8, device="cuda")
        dw = torch.full((E, N, K), 77.0, dtype=torch.bfloat16, device="cuda")
        B.moe_grouped_linear_fp8_wgrad(g, u8(nb * 128, K), one(nb, 1), u8(nb * 128, N), one(nb, N),
                                       torch.tensor(split, dtype=torch.int32, device="cuda"), dw, ws)
        assert B.moe_get_device_error(ws)[0] == code and bool((dw == want).all())


def test_cut_weight_gradients_in_two_graphs():
    """Two graphs that share a workspace, replayed in turn with other rows: each gives what its eager call gives."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    cases = []
    for split, K, N in (([9000, 100], 256, 144), ([50, 5000, 3], 64, 528)):
        R, E = sum(split), len(split)
        g, nb = B.grouped(R, K, N, E), B.fp8_blocks(R, E)
        code = lambda c: torch.randint(0, 100, (nb * 128, c), generator=gen, device="cuda").to(torch.uint8)  # noqa: B023,E731
        cases.append([g, code(K), torch.rand(nb, -(-K // 128), generator=gen, device="cuda"), code(N),
                      torch.rand(nb, N, generator=gen, device="cuda"), torch.tensor(split, dtype=torch.int32, device="cuda"),
                      torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda")])
    ws = torch.zeros(max(B.moe_grouped_linear_fp8_workspace_size(c[0]) for c in cases), dtype=torch.uint8, device="cuda")
    want, graphs = [], []
    for c in cases:
        B.moe_grouped_linear_fp8_wgrad(*c, ws)
        want.append(c[-1].clone())
    for c in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            B.moe_grouped_linear_fp8_wgrad(*c, ws)
    for i in (0, 1, 1, 0, 1):
        cases[i][-1].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(cases[i][-1], want[i])
    assert B.moe_get_device_error(ws) == (0, 0)


def test_rows_past_the_sum_and_pitches():
    check_whole([40, 0, 9], 96, 112, rows=300, seed=4, pad=24)
    check_whole([40, 0, 9], 96, 112, rows=300, seed=5, pad=16)


def test_one_row_does_not_reach_another():
    """NaN in a row (its codes, or its scale) stays in that row's y and dx; in an expert's block of tokens, in that
    expert's dw."""
    split, K, N = [21, 45, 30], 144, 80
    c = Case(split, K, N, 100, 9, True)
    clean = c.run()
    for k in ("x", "dy"):
        c.dev[k][22] = 0x7F                                  # a row of expert 1
        c.dev[k][97:] = 0x7F                                 # rows of no expert
    c.dev["xs"][:, 23] = float("nan")
    c.dev["dyt"][128 + 1] = 0x7F                             # expert 1's second row
    y, dx, dw = c.run()
    others = [i for i in range(96) if i not in (22, 23)]
    assert torch.equal(y[others], clean[0][others]) and bool(y[22:24].isnan().all())
    assert torch.equal(dx[others], clean[1][others]) and bool(dx[22].isnan().all()) and torch.equal(dx[23], clean[1][23])
    assert torch.equal(dw[0], clean[2][0]) and torch.equal(dw[2], clean[2][2]) and bool(dw[1].isnan().all())


@pytest.mark.parametrize("split", [[5, -1, 4], [5, 60, 4], [2 ** 30, 2 ** 30, 2 ** 30]])
def test_inconsistent_sizes_are_recorded_and_write_nothing(split):
    c = Case([5, 3, 4], 64, 64, 40, 1, True)
    ss, d = torch.tensor(split, dtype=torch.int32, device="cuda"), c.dev
    for op in range(3):
        ws = torch.zeros_like(c.ws)
        out = torch.full((3, 64, 64) if op == 2 else (40, 64), 77.0, dtype=torch.bfloat16, device="cuda")
        if op == 0:
            B.moe_grouped_linear_fp8_fwd(c.g, d["x"], d["xs"], ss, d["w"], d["ws"], out, ws)
        elif op == 1:
            B.moe_grouped_linear_fp8_dgrad(c.g, d["dy"], d["dys"], ss, d["w"], d["ws"], out, ws)
        else:
            B.moe_grouped_linear_fp8_wgrad(c.g, d["xt"], d["xts"], d["dyt"], d["dyts"], ss, out, ws)
        assert B.moe_get_device_error(ws)[0] == 7
        assert bool((out == 77.0).all())


def test_no_rows():
    c = Case([0, 0, 0], 64, 64, 0, 1, True)
    y, dx, dw = c.run()
    assert y.numel() == 0 and dx.numel() == 0 and not bool(dw.any())


@pytest.mark.parametrize("rows,K,N", [(1, 64, 64), (40, 1040, 528), (3000, 256, 144)])
def test_rows_but_no_expert_has_any(rows, K, N):
    c = Case([0, 0, 0], K, N, rows, 2, True)
    y, dx, dw = c.run()                                      # (checks that no row is written)
    assert not bool(dw.any())


def test_reproducible():
    c = Case([100, 33, 250], 272, 528, 383, 6, False)
    for a, b in zip(c.run(), c.run()):
        assert torch.equal(a, b)
