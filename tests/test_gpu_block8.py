"""Fp8MoEBlock (root-mean-square norm with 8-bit rows, router, balance loss, grouped linears on 8-bit operands)
against float64.

The oracle follows the device's expert choices and its kept codes (both checked against its own), quantizes where
the block does, and rounds to bf16 where the block stores bf16 tensors.  What remains are values that fall on the
other side of a rounding: a bf16 value that is off by 2^-8 and happens to be its block's largest moves that
block's 8-bit codes by up to half a step (2^-4 / sqrt(3) = 0.036 of them, root mean square), which a few blocks in a
thousand do: bound 0.01, as for the block of bf16 products.
"""
import numpy as np
import pytest
import torch

from helpers import rel_frob
from moe_expert_ffn_03_gb300 import binding as B, build
from moe_expert_ffn_03_gb300.block8 import Fp8MoEBlock, Scratch8, Weights8
from oracle import block as bl
from oracle import fp8_block as fb
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
    return {"gamma": (torch.rand(H, generator=g, device="cuda") + 0.5).bfloat16(), "w_r": mk(E, H, std=0.05),
            "w_gu": Weights8(E, 2 * I, H).quantize(mk(E, 2 * I, H, std=0.05)),
            "w_d": Weights8(E, H, I).quantize(mk(E, H, I, std=0.05))}


def values(w8):
    return np.stack([fb.tiles_back(c, s) for c, s in zip(w8.codes.cpu().numpy(), w8.scales.cpu().numpy())])


def rows8(v):
    return fb.rows_back(*fb.rows8(v))


def along_tokens(v, split, tiles):
    """v's rows as their values along tokens are, without the rows behind the experts' last."""
    back = (fb.tiles_back if tiles else fb.tokens_back)(*fb.tokens8(v, split, tiles))
    first, _ = fb.layout(split)
    return np.concatenate([back[f: f + n] for f, n in zip(first, split)])


def check(blk, x, residual, w, h, out, dout, dx, mask=None, dloss=1.0):
    T, H, I, E, k = blk.T, blk.H, blk.I, blk.E, blk.k
    gamma, w_r, w_gu, w_d = f64(w["gamma"]), f64(w["w_r"]), values(w["w_gu"]), values(w["w_d"])
    x64 = f64(x) + (f64(residual) if residual is not None else 0.0)
    n, _, _ = fb.rmsnorm(x64, gamma, 1e-5)
    n8 = fb.rows_back(blk.n_codes.cpu().numpy(), blk.n_scales.cpu().numpy())
    assert rel_frob(n8, n) < 0.04
    logits = ro.router_logits(mx.bf16(n), w_r, rounded=False)
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
    gu = mx.bf16(bl.grouped_linear(n8[tok], w_gu, split))
    a = mx.bf16(bl.swiglu(gu[:, :I], gu[:, I:], p))
    y = mx.bf16(bl.grouped_linear(rows8(a), w_d, split))
    assert rel_frob(f64(h), x64) < BOUND and rel_frob(f64(out), y[pos].reshape(T, k, H).sum(1)) < BOUND
    aux = 0.0
    if blk.balanced:
        alpha, beta = blk.loss_of.alpha, blk.loss_of.beta
        counts, live, mean, loss, aux = fb.balance(logits, idx, alpha, beta, None if mask is None else mask.cpu().numpy())
        assert np.array_equal(blk.counts.cpu().numpy(), np.concatenate([counts, [live]]))
        assert rel_frob(blk.prob_mean.cpu().numpy(), mean) < BOUND and rel_frob(blk.loss.cpu().numpy(), np.array(loss)) < BOUND
    if not blk.training:
        return
    # backward, from the device's kept codes
    nb = (I + 31) // 32
    codes, scales = blk.gu_codes.cpu().numpy(), blk.gu_scales.cpu().numpy()
    g8, u8 = bl.act8_decode(codes[:, :I], scales[:, :nb]), bl.act8_decode(codes[:, I:], scales[:, nb:])
    assert rel_frob(np.concatenate([g8, u8], 1), gu) < 0.04
    do = f64(dout)
    dy = do[tok]
    da = mx.bf16(bl.grouped_linear_dgrad(rows8(dy), w_d, split))
    dg, du, dp = bl.swiglu_backward(g8, u8, p, da)
    dgu = mx.bf16(np.concatenate([dg, du], 1))
    a_back = along_tokens(mx.bf16(bl.swiglu(g8, u8, p)), split, True)
    assert rel_frob(f64(blk.dw_d), bl.grouped_linear_wgrad(a_back, along_tokens(dy, split, False), split)) < BOUND
    n16 = mx.bf16(n8)
    assert rel_frob(f64(blk.dw_gu), bl.grouped_linear_wgrad(along_tokens(n16[tok], split, True), along_tokens(dgu, split, False), split)) < BOUND
    dn = mx.bf16(mx.bf16(bl.grouped_linear_dgrad(rows8(dgu), w_gu, split))[pos].reshape(T, k, H).sum(1))
    dl = ro.router_backward(logits, idx, prob, dp[pos].reshape(T, k)) + aux * dloss
    dn_r, dw_r = ro.router_input_grads(dl, n16, w_r)
    assert rel_frob(f64(blk.dw_r), dw_r) < BOUND
    h64 = f64(h)
    _, norm, rstd = fb.rmsnorm(h64, gamma, 1e-5)
    rdx, rdg = fb.rmsnorm_backward(ro.add_to_bf16(dn, dn_r), norm, rstd, gamma, do)
    assert rel_frob(f64(dx), rdx) < BOUND and rel_frob(f64(blk.dgamma), rdg) < BOUND
    assert blk.device_error() == (0, 0)


def tensors(T, H, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    mk = lambda std: (torch.randn(T, H, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    return g, mk(1.0), mk(0.5), mk(0.1)


@pytest.mark.parametrize("T,H,I,E,k", [(300, 256, 384, 8, 2), (1, 128, 128, 4, 2), (129, 384, 128, 16, 4), (700, 128, 256, 4, 3)])
@pytest.mark.parametrize("with_residual", [False, True])
def test_block(T, H, I, E, k, with_residual):
    g, x, residual, dout = tensors(T, H, T + E)
    w = weights(H, I, E, g)
    blk = Fp8MoEBlock(T, H, I, E, k)
    residual = residual if with_residual else None
    h, out = blk.forward(x, w, residual)
    dx = blk.backward(dout, w)
    check(blk, x, residual, w, h, out, dout, dx)


@pytest.mark.parametrize("masked", [False, True])
def test_balance_loss(masked):
    T, H, I, E, k = 260, 256, 128, 8, 2
    g, x, residual, dout = tensors(T, H, 5)
    w = weights(H, I, E, g)
    mask = (torch.rand(T, generator=g, device="cuda") < 0.7).to(torch.uint8) if masked else None
    blk = Fp8MoEBlock(T, H, I, E, k, alpha=30.0, beta=3.0)
    h, out = blk.forward(x, w, residual, mask)
    dloss = torch.tensor([0.75], device="cuda")
    dx = blk.backward(dout, w, dloss)
    check(blk, x, residual, w, h, out, dout, dx, mask, 0.75)
    # what it adds to the logits' gradient is the formula's, to the rounding of the float32 sum and 2^-17 (some ten
    # roundings, exp and log among them) of its own terms, of which a token's largest stands for all
    plain = Fp8MoEBlock(T, H, I, E, k)
    plain.forward(x, w, residual)
    plain.backward(dout, w)
    with_it, without = f64(blk.s.dlogits), f64(plain.s.dlogits)
    aux = 0.75 * fb.balance(f64(blk.logits), blk.idx.cpu().numpy(), 30.0, 3.0, None if mask is None else mask.cpu().numpy())[4]
    bound = 2.0 ** -23 * (np.abs(with_it) + np.abs(without)) + 2.0 ** -17 * np.abs(aux).max(1, keepdims=True)
    assert np.abs(aux).max() > 0 and np.all(np.abs(with_it - without - aux) <= bound)


def test_inference():
    T, H, I, E, k = 33, 256, 128, 8, 2
    g, x, residual, dout = tensors(T, H, 7)
    w = weights(H, I, E, g)
    blk, full = Fp8MoEBlock(T, H, I, E, k, training=False), Fp8MoEBlock(T, H, I, E, k)
    h, out = blk.forward(x, w, residual)
    check(blk, x, residual, w, h, out, dout, None)
    h2, out2 = full.forward(x, w, residual)
    assert torch.equal(h, h2) and torch.equal(out, out2)
    with pytest.raises(RuntimeError, match="inference"):
        blk.backward(dout, w)


def test_blocks_share_scratch():
    """Two blocks in a row on one set of scratch buffers: the second's passes leave what the first kept untouched."""
    T, H, I, E, k = 200, 256, 256, 8, 2
    g, x, _, dout = tensors(T, H, 3)
    s = Scratch8(T, H, I, E, k)
    first, second = Fp8MoEBlock(T, H, I, E, k, scratch=s), Fp8MoEBlock(T, H, I, E, k, scratch=s)
    w1, w2 = weights(H, I, E, g), weights(H, I, E, g)
    h1, out1 = first.forward(x, w1)
    h2, out2 = second.forward(h1, w2, residual=out1)
    d2 = second.backward(dout, w2).clone()
    d1 = first.backward(d2, w1)
    check(second, h1, out1, w2, h2, out2, dout, d2)
    check(first, x, None, w1, h1, out1, d2, d1)


def test_recorded_in_a_graph():
    """A training step replayed on refilled inputs gives the eager step's results bit for bit."""
    T, H, I, E, k = 96, 256, 128, 8, 2
    g, x, residual, dout = tensors(T, H, 9)
    w = weights(H, I, E, g)
    blk = Fp8MoEBlock(T, H, I, E, k, alpha=0.1, beta=0.01)

    def run():
        blk.forward(x, w, residual)
        blk.backward(dout, w)

    outs = lambda: [t.clone() for t in (blk.h, blk.out, blk.loss, blk.counts, blk.dx, blk.dgamma, blk.dw_r, blk.dw_gu, blk.dw_d)]  # noqa: E731
    fills = [[t.clone() for t in (x, residual, dout)], [t.roll(1, 0) * 0.5 for t in (dout * 8, x, residual)]]

    def fill(i):
        for t, v in zip((x, residual, dout), fills[i]):
            t.copy_(v)

    want = []
    for i in (0, 1):
        fill(i)
        run()
        want.append(outs())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in (1, 0, 1):
        fill(i)
        for t in (blk.out, blk.dx, blk.dw_gu, blk.dw_d):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs(), want[i]))
    assert not torch.equal(want[0][4], want[1][4]) and blk.device_error() == (0, 0)


def test_on_another_stream():
    T, H, I, E, k = 96, 256, 128, 8, 2
    g, x, residual, dout = tensors(T, H, 11)
    w = weights(H, I, E, g)
    blk = Fp8MoEBlock(T, H, I, E, k, alpha=0.1)
    blk.forward(x, w, residual)
    want = blk.backward(dout, w).clone()
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    blk.dx.zero_()
    with torch.cuda.stream(other):
        blk.forward(x, w, residual)
        got = blk.backward(dout, w)
    other.synchronize()
    assert torch.equal(got, want)
