"""MoEBlock (norm, router, grouped linears, gated activation, 8-bit checkpoints) against float64.

The oracle follows the device's expert choices and, in the backward, its kept codes (both checked
against its own), and rounds to bf16 where the block stores bf16 tensors (a difference of two
tokens' terms, as in the router's gradient, carries those roundings whole).  What remains are values
that fall on the other side of a rounding; bound 0.01, two to three roundings of 2^-8.
"""
import numpy as np
import pytest
import torch

from helpers import rel_frob
from moe_expert_ffn_03_gb300 import binding as B, build, configs, synth
from moe_expert_ffn_03_gb300.block import MoEBlock, Scratch
from moe_expert_ffn_03_gb300.layer import ExpertFFN
from oracle import block as bl
from oracle import mxfp8 as mx
from oracle import router as ro
from oracle import routing as rt
from rowcheck import f64

pytestmark = pytest.mark.gpu
BOUND = 1e-2


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def weights(H, I, E, g):
    mk = lambda *s, std: (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    return {"gamma": (torch.rand(H, generator=g, device="cuda") + 0.5).bfloat16(), "beta": mk(H, std=0.1),
            "w_r": mk(E, H, std=0.05), "w_gu": mk(E, 2 * I, H, std=0.05), "w_d": mk(E, H, I, std=0.05)}


def check(blk, x, residual, w, h, out, dout, dx):
    T, H, I, E, k = blk.T, blk.H, blk.I, blk.E, blk.k
    W = {n: f64(v) for n, v in w.items()}
    x64 = f64(x) + (f64(residual) if residual is not None else 0.0)
    n, norm, _, rstd = bl.layernorm(x64, W["gamma"], W["beta"], 1e-5)
    n = mx.bf16(n)
    logits = ro.router_logits(n, W["w_r"], rounded=False)
    idx = blk.idx.cpu().numpy()
    mine, _ = rt.route_topk(logits.astype(np.float32), k)
    ranked = np.sort(logits, axis=1)[:, ::-1]
    gap = ranked[:, k - 1] - ranked[:, k] if E > k else np.ones(T)
    sure = gap > 0.02                    # n is rounded to bf16 on both sides, now and then apart
    assert all(set(a) == set(b) for a, b in zip(mine[sure], idx[sure]))
    prob = ro.probs_from_logits(logits, idx)
    order = np.argsort(idx.reshape(-1), kind="stable")            # rows by expert, tokens in order
    split = np.bincount(idx.reshape(-1), minlength=E)
    assert np.array_equal(blk.split_sizes.cpu().numpy(), split)
    pos = np.empty(T * k, dtype=int)
    pos[order] = np.arange(T * k)
    assert np.array_equal(blk.pos_of.cpu().numpy().reshape(-1), pos)
    tok, p = order // k, prob.reshape(-1)[order]
    gu = mx.bf16(bl.grouped_linear(n[tok], W["w_gu"], split))
    a = mx.bf16(bl.swiglu(gu[:, :I], gu[:, I:], p))
    y = mx.bf16(bl.grouped_linear(a, W["w_d"], split))
    assert rel_frob(f64(h), x64) < BOUND and rel_frob(f64(out), y[pos].reshape(T, k, H).sum(1)) < BOUND
    # backward, from the device's kept codes (each within half an E4M3 step of the oracle's value)
    nb = (I + 31) // 32
    codes, scales = blk.gu_codes.cpu().numpy(), blk.gu_scales.cpu().numpy()
    g8, u8 = bl.act8_decode(codes[:, :I], scales[:, :nb]), bl.act8_decode(codes[:, I:], scales[:, nb:])
    assert rel_frob(np.concatenate([g8, u8], 1), gu) < 0.04
    norm8 = bl.act8_decode(blk.n_codes.cpu().numpy(), blk.n_scales.cpu().numpy())
    assert rel_frob(norm8, norm) < 0.04
    n8 = mx.bf16(norm8 * W["gamma"] + W["beta"])
    do = f64(dout)
    dy = do[tok]
    da = mx.bf16(bl.grouped_linear_dgrad(dy, W["w_d"], split))
    dg, du, dp = bl.swiglu_backward(g8, u8, p, da)
    dgu = mx.bf16(np.concatenate([dg, du], 1))
    assert rel_frob(f64(blk.dw_d), bl.grouped_linear_wgrad(mx.bf16(bl.swiglu(g8, u8, p)), dy, split)) < BOUND
    assert rel_frob(f64(blk.dw_gu), bl.grouped_linear_wgrad(n8[tok], dgu, split)) < BOUND
    dn = mx.bf16(mx.bf16(bl.grouped_linear_dgrad(dgu, W["w_gu"], split))[pos].reshape(T, k, H).sum(1))
    dl = ro.router_backward(logits, idx, prob, dp[pos].reshape(T, k))
    dn_r, dw_r = ro.router_input_grads(dl, n8, W["w_r"])
    assert rel_frob(f64(blk.dw_r), dw_r) < BOUND
    rdx, rdg, rdb = bl.layernorm_backward(ro.add_to_bf16(dn, dn_r), norm8, rstd, W["gamma"], do)
    assert rel_frob(f64(dx), rdx) < BOUND and rel_frob(f64(blk.dgamma), rdg) < BOUND and rel_frob(f64(blk.dbeta), rdb) < BOUND
    assert blk.device_error() == (0, 0)


@pytest.mark.parametrize("T,H,I,E,k", [(300, 256, 384, 8, 2), (1, 128, 128, 4, 2), (129, 384, 128, 16, 4)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_block(T, H, I, E, k, with_residual):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    mk = lambda std: (torch.randn(T, H, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    w = weights(H, I, E, g)
    blk = MoEBlock(T, H, I, E, k)
    x, residual, dout = mk(1.0), mk(0.5) if with_residual else None, mk(0.1)
    h, out = blk.forward(x, w, residual)
    dx = blk.backward(dout, w)
    check(blk, x, residual, w, h, out, dout, dx)


def test_blocks_share_scratch():
    """Two blocks in a row on one set of scratch buffers: the second's passes leave what the first
    kept untouched.  Per layer that is less than half of what bf16 tensors would take."""
    T, H, I, E, k = 200, 256, 256, 8, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    mk = lambda std: (torch.randn(T, H, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    s = Scratch(T, H, I, E, k)
    first, second = MoEBlock(T, H, I, E, k, scratch=s), MoEBlock(T, H, I, E, k, scratch=s)
    w1, w2 = weights(H, I, E, g), weights(H, I, E, g)
    x, dout = mk(1.0), mk(0.1)
    h1, out1 = first.forward(x, w1)
    h2, out2 = second.forward(h1, w2, residual=out1)
    d2 = second.backward(dout, w2).clone()
    d1 = first.backward(d2, w1)
    check(second, h1, out1, w2, h2, out2, dout, d2)
    check(first, x, None, w1, h1, out1, d2, d1)
    assert second.kept_bytes() < 0.56 * 2 * (T * H + T * k * 2 * I)


def test_saved_gate_and_up_in_8_bits():
    """ExpertFFN's saved g and u through an 8-bit checkpoint between its passes: dx moves by the
    checkpoint's error and not more (an E4M3 step is 2^-3 of a value at most, so a uniform error
    2^-4 / sqrt(3) = 0.036 at most, and the gradients are sums of such terms)."""
    wl = configs.small(300, 256, 256, 8, 2, backward=True)
    inp = {n: v.cuda() for n, v in synth.make_inputs(wl, 0).items()}
    L = ExpertFFN(wl.T, wl.H, wl.I, wl.E, wl.k, training=True)
    L.quantize_weights(inp["w_gu"], inp["w_d"])
    L.forward(inp["logits"], inp["x"])
    dx = L.backward(inp["dout"]).clone()
    dw = L.dwgu.clone()
    rows, cols = L.saved_gu.shape
    L.saved_gu[L.padded_rows():] = 0                        # rows that no call has written
    codes = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, cols // 32, dtype=torch.uint8, device="cuda")
    B.moe_act8_pack(L.saved_gu, codes, scales)
    L.saved_gu.zero_()                                      # other layers' passes use the buffer meanwhile
    B.moe_act8_unpack(codes, scales, None, None, L.saved_gu)
    dx8 = L.backward(inp["dout"])
    assert 0 < rel_frob(f64(dx8), f64(dx)) < 0.072 and 0 < rel_frob(f64(L.dwgu), f64(dw)) < 0.072
