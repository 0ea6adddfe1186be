"""Tensors past 2^31 elements, calls side by side on two streams: the operators on blocks of 128."""
import numpy as np
import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build
from oracle import fp8_block as fb
from rowcheck import f64

pytestmark = pytest.mark.gpu
BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    yield
    torch.cuda.empty_cache()


def new(*s, dt=BF16, fill=0):
    return torch.full(s, fill, dtype=dt, device="cuda")


def some(rows, n=40):
    """The first, the last and some rows between."""
    return sorted({0, 1, rows - 1, rows - 2, *np.random.default_rng(0).integers(0, rows, n).tolist()})


def test_quantize_and_back():
    R, C = 1_100_003, 2048                                   # 2.25e9 values
    split = [R - 5, 0, 5]
    v = torch.randn(R, C, device="cuda", dtype=BF16)
    nb = B.fp8_blocks(R, 3)
    c, s, tc, ts = new(R, C, dt=U8), new(C // 128, R, dt=F32), new(nb * 128, C, dt=U8), new(nb, C, dt=F32)
    B.moe_fp8_block_quantize(v, c, s, torch.tensor(split, dtype=I32, device="cuda"), tc, ts)
    at = some(R)
    rc, rs = fb.rows8(v[at].float().cpu().numpy())
    assert np.array_equal(c[at].cpu().numpy(), rc) and np.array_equal(s[:, at].cpu().numpy(), rs)
    first, _ = fb.layout(split)
    last = v[R - 5:].float().cpu().numpy()
    rc, rs = fb.tokens8(last, [5], False)
    assert np.array_equal(tc[first[2]: first[2] + 128].cpu().numpy(), rc) and np.array_equal(ts[first[2] // 128][None].cpu().numpy(), rs)
    blk = (R - 5) // 128 - 1                                 # the last full block of the first expert
    rc, rs = fb.tokens8(v[blk * 128: blk * 128 + 128].float().cpu().numpy(), [128], False)
    assert np.array_equal(tc[blk * 128: blk * 128 + 128].cpu().numpy(), rc) and np.array_equal(ts[blk][None].cpu().numpy(), rs)
    del tc, ts
    out = new(R, C)
    B.moe_fp8_block_dequantize(c, s, "rows", out)
    rc, rs = fb.rows8(v[at].float().cpu().numpy())
    assert torch.equal(out[at].cpu(), torch.tensor(fb.rows_back(rc, rs)).float().bfloat16())


def test_rmsnorm():
    R, H = 270_001, 8192                                     # 2.2e9 values
    x, gamma = torch.randn(R, H, device="cuda", dtype=BF16), torch.ones(H, device="cuda", dtype=BF16)
    n = B.norm(R, H)
    y, rstd, c, s = new(R, H), new(R, dt=F32), new(R, H, dt=U8), new(H // 128, R, dt=F32)
    B.moe_rmsnorm_fwd(n, x, None, gamma, None, y, rstd, c, s)
    at = some(R, 10)
    ry, _, rr = fb.rmsnorm(f64(x[at]), np.ones(H), float(np.float32(1e-5)))
    e = (H / 64 + 12) * 2.0 ** -24
    assert np.allclose(f64(rstd[at]), rr, rtol=e, atol=0)
    assert np.all(np.abs(f64(y[at]) - ry) <= np.abs(ry) * (2.0 ** -8 * 1.01 + e))
    back = fb.rows_back(c[at].cpu().numpy(), s[:, at].cpu().numpy())
    assert np.all(np.abs(back - ry) <= np.maximum(np.abs(ry) / 16, np.abs(ry).max() / 448 * 2.0 ** -10) * (1 + 1e-4) + 1e-6)
    dx, dg = new(R, H), new(H)
    ws = new(B.moe_rmsnorm_workspace_size(n), dt=U8)
    B.moe_rmsnorm_bwd(n, y, x, rstd, gamma, None, dx, dg, ws)     # the gradient is y: dx = rstd (y - n mean(y n)) is near 0
    n64 = f64(x[at]) * f64(rstd[at])[:, None]
    rdx, _ = fb.rmsnorm_backward(f64(y[at]), n64, f64(rstd[at]), np.ones(H))
    assert np.all(np.abs(f64(dx[at]) - rdx) <= 2.0 ** -8 * np.abs(rdx) + np.abs(f64(rstd[at]))[:, None] * np.abs(n64) * (H / 32 + 20) * 2.0 ** -24 + 1e-6)


@pytest.mark.parametrize("split,K,N", [([140_000, 0, 1003], 128, 16384), ([1_100_000, 77], 2048, 16)])
def test_grouped_linear(split, K, N):
    """Outputs, or operands, of more than 2^31 values.  Codes of -1, 0 and 1: sums of at most 2048
    such products, of variance 0.44, stay below 2^8 (eight standard deviations), where bf16 holds whole numbers."""
    R, E = sum(split), len(split)
    g = B.grouped(R, K, N, E)
    ss = torch.tensor(split, dtype=I32, device="cuda")
    ws = new(B.moe_grouped_linear_fp8_workspace_size(g), dt=U8)
    pick = torch.tensor([0x38, 0xB8, 0], dtype=U8, device="cuda")
    draw = lambda *s: pick[torch.randint(0, 3, s, device="cuda", dtype=torch.uint8).int()] if np.prod(s) < 2 ** 28 else torch.cat([draw(s[0] // 8 + (i < s[0] % 8), *s[1:]) for i in range(8)])  # noqa: E731
    x, w = draw(R, K), draw(E, N, K)
    one = lambda *s: new(*s, dt=F32, fill=1)  # noqa: E731
    cut = lambda n: -(-n // 128)  # noqa: E731
    y = new(R, N, fill=77)
    B.moe_grouped_linear_fp8_fwd(g, x, one(cut(K), R), ss, w, one(E, cut(N), cut(K)), y, ws)
    assert B.moe_get_device_error(ws) == (0, 0)
    at = some(R)
    owner = np.searchsorted(np.cumsum(split), at, side="right")
    xv, wv = fb.E4M3[x[at].cpu().numpy()], fb.E4M3[w.cpu().numpy()]
    for r, i, e in zip(range(len(at)), at, owner):
        assert np.array_equal(f64(y[i]), xv[r] @ wv[e].T), i


def test_weight_gradient():
    """2.7e9 outputs, of experts without rows and with few."""
    E, N, K = 40, 8192, 8192
    split = [0] * E
    split[3], split[E - 1] = 130, 7
    R = sum(split)
    g, nb = B.grouped(R, K, N, E), B.fp8_blocks(R, E)
    ss = torch.tensor(split, dtype=I32, device="cuda")
    ws = new(B.moe_grouped_linear_fp8_workspace_size(g), dt=U8)
    xt, dyt = new(nb * 128, K, dt=U8), new(nb * 128, N, dt=U8)
    first, _ = fb.layout(split)
    gen = torch.Generator(device="cuda").manual_seed(0)
    for e in (3, E - 1):
        for t in (xt, dyt):
            t[first[e]: first[e] + split[e]] = torch.where(torch.rand(split[e], t.shape[1], generator=gen, device="cuda") < 0.5, 0x38, 0xB8).to(U8)
    dw = new(E, N, K, fill=77)
    B.moe_grouped_linear_fp8_wgrad(g, xt, new(nb, K // 128, dt=F32, fill=1), dyt, new(nb, N, dt=F32, fill=1), ss, dw, ws)
    assert B.moe_get_device_error(ws) == (0, 0)
    rows = some(N, 6)
    for e in range(E):
        a = slice(int(first[e]), int(first[e]) + split[e])
        ref = fb.E4M3[dyt[a].cpu().numpy()][:, rows].T @ fb.E4M3[xt[a].cpu().numpy()]
        assert np.array_equal(f64(dw[e][rows]), ref), e
        assert split[e] or not bool(dw[e].any())


def test_calls_side_by_side():
    """Two streams, a workspace each: the calls may run at the same time and give what they give alone."""
    R, K, N, E = 24, 2048, 1024, 4
    g = B.grouped(R, K, N, E)
    ss = torch.tensor([5, 7, 0, 12], dtype=I32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    code = lambda *s: torch.randint(0, 120, s, generator=gen, device="cuda", dtype=torch.int32).to(U8)  # noqa: E731
    w, sw = code(E, N, K), torch.rand(E, N // 128, K // 128, generator=gen, device="cuda")
    xs = [(code(R, K), torch.rand(K // 128, R, generator=gen, device="cuda")) for _ in range(2)]
    logits = [torch.randn(4000, 64, generator=gen, device="cuda") for _ in range(2)]
    idx = [x.topk(6, 1).indices.to(I32) for x in logits]
    b = B.balance(4000, 64, 6, 0.1, 0.1)

    def state(i):
        return {"ws": new(B.moe_grouped_linear_fp8_workspace_size(g), dt=U8), "wb": new(B.moe_balance_loss_workspace_size(b), dt=U8),
                "y": new(R, N), "counts": new(65, dt=I32), "prob": new(64, dt=F32), "loss": new(3, dt=F32), "dl": new(4000, 64, dt=F32)}

    def go(i, s, stream=None):
        B.moe_grouped_linear_fp8_fwd(g, *xs[i], ss, w, sw, s["y"], s["ws"], stream)
        B.moe_balance_loss_fwd(b, logits[i], idx[i], None, s["counts"], s["prob"], s["loss"], s["wb"], stream)
        B.moe_balance_loss_bwd(b, logits[i], None, s["counts"], None, s["dl"], stream)

    want = [state(0), state(1)]
    for i in range(2):
        go(i, want[i])
    got, streams = [state(0), state(1)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            go(i, got[i], streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        for k in ("y", "counts", "prob", "loss", "dl"):
            assert torch.equal(got[i][k], want[i][k]), k
