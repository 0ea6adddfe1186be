"""The operators around the layer in CUDA graphs: what one token of a served model, or a training step of
small blocks, is recorded as.  A replay gives the eager calls' results bit for bit, also on refilled inputs."""
import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build
from moe_expert_ffn_03_gb300.block import MoEBlock

pytestmark = pytest.mark.gpu
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def check(run, outputs, fill):
    """run() on its own and recorded; fill(seed) refills the inputs in place."""
    def eager(seed):
        fill(seed)
        for t in outputs:
            t.zero_()
        run()
        return [t.clone() for t in outputs]

    want = {seed: eager(seed) for seed in (1, 2)}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in (2, 1, 2):
        fill(seed)
        for t in outputs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outputs, want[seed]):
            assert torch.equal(got, ref)
    assert not any(torch.equal(a, b) for a, b in zip(want[1], want[2])), "the inputs do not change the results"


def filler(tensors, scale=1.0):
    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        for t in tensors:
            t.copy_(torch.randn(t.shape, generator=g, device="cuda") * scale)
    return fill


def new(*s, dt=BF16):
    return torch.zeros(*s, dtype=dt, device="cuda")


@pytest.mark.parametrize("rows,H,act8", [(1, 1024, False), (1, 1001, True), (300, 264, True)])
def test_layernorm(rows, H, act8):
    n = B.norm(rows, H)
    x, gamma, beta, dy = new(rows, H), new(H), new(H), new(rows, H)
    y, mean, rstd, dx, dg, db = new(rows, H), new(rows, dt=F32), new(rows, dt=F32), new(rows, H), new(H), new(H)
    codes, scales = (new(rows, H, dt=U8), new(rows, (H + 31) // 32, dt=U8)) if act8 else (None, None)
    ws = new(B.moe_layernorm_workspace_size(n), dt=U8)

    def run():
        B.moe_layernorm_fwd(n, x, None, gamma, beta, None, y, mean, rstd, codes, scales)
        B.moe_layernorm_bwd(n, dy, None if act8 else x, mean, rstd, codes, scales, gamma, None, dx, dg, db, ws)

    check(run, [y, mean, rstd, dx, dg, db], filler([x, gamma, beta, dy]))


@pytest.mark.parametrize("rows,I", [(2, 1408), (12, 1001), (500, 256)])
def test_gated_activation_and_act8(rows, I):
    gu, prob, da, back = new(rows, 2 * I), new(rows, dt=F32), new(rows, I), new(rows, 2 * I)
    a, a2, dgu, dp = new(rows, I), new(rows, I), new(rows, 2 * I), new(rows, dt=F32)
    codes, scales = new(rows, 2 * I, dt=U8), new(rows, 2 * ((I + 31) // 32), dt=U8)
    c2, s2 = new(rows, 2 * I, dt=U8), new(rows, (2 * I + 31) // 32, dt=U8)

    def run():
        B.moe_swiglu_fwd(gu, prob, a, codes, scales)
        B.moe_swiglu_bwd(None, codes, scales, prob, da, dgu, dp, a2)
        B.moe_act8_pack(gu, c2, s2)
        B.moe_act8_unpack(c2, s2, None, None, back)

    check(run, [a, a2, dgu, dp, back], filler([gu, prob, da]))


@pytest.mark.parametrize("split,K,N", [([1, 1], 2048, 1024), ([0, 0, 7, 0], 136, 264), ([200, 33, 90], 256, 512)])
def test_grouped_linear(split, K, N):
    R, E = sum(split), len(split)
    g, ss = B.grouped(R, K, N, E), torch.tensor(split, dtype=torch.int32, device="cuda")
    x, dy, w, y, dx, dw = new(R, K), new(R, N), new(E, N, K), new(R, N), new(R, K), new(E, N, K)
    ws = new(B.moe_grouped_linear_workspace_size(g), dt=U8)

    def run():
        B.moe_grouped_linear_fwd(g, x, ss, w, y, ws)
        B.moe_grouped_linear_dgrad(g, dy, ss, w, dx, ws)
        B.moe_grouped_linear_wgrad(g, x, dy, ss, dw, ws)

    check(run, [y, dx, dw], filler([x, dy, w]))
    assert B.moe_get_device_error(ws) == (0, 0)


@pytest.mark.parametrize("T", [1, 130])
def test_block(T):
    H, I, E, k = 256, 128, 8, 2
    blk = MoEBlock(T, H, I, E, k)
    w = {"gamma": new(H), "beta": new(H), "w_r": new(E, H), "w_gu": new(E, 2 * I, H), "w_d": new(E, H, I)}
    x, res, dout = new(T, H), new(T, H), new(T, H)

    def run():
        blk.forward(x, w, res)
        blk.backward(dout, w)

    check(run, [blk.h, blk.out, blk.dx, blk.dgamma, blk.dbeta, blk.dw_r, blk.dw_gu, blk.dw_d],
          filler([x, res, dout, *w.values()], 0.5))
    assert blk.device_error() == (0, 0)
