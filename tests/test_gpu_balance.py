"""The balance loss on the device against float64.

Every softmax entry takes some ten float32 operations of relative error 2^-24 (exp's and log's few units among
them: 2^-22 each), a sum of n tokens at most n / 64 + 40 additions behind any term; a gradient entry is the
difference of two such terms, each with 2^-19 of its own size.
"""
import numpy as np
import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build
from oracle import fp8_block as fb

pytestmark = pytest.mark.gpu

ALPHA, BETA = 0.013, 0.0021


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def run(logits, idx, mask=None, grad=None, alpha=ALPHA, beta=BETA, ws=None):
    T, E = logits.shape
    b = B.balance(T, E, idx.shape[1], alpha=alpha, beta=beta)
    if ws is None:
        ws = torch.zeros(B.moe_balance_loss_workspace_size(b), dtype=torch.uint8, device="cuda")
    counts = torch.full((E + 1,), 77, dtype=torch.int32, device="cuda")
    prob, loss = torch.full((E,), 77.0, device="cuda"), torch.full((3,), 77.0, device="cuda")
    dl = torch.full((T, E), 77.0, device="cuda")
    B.moe_balance_loss_fwd(b, logits, idx, mask, counts, prob, loss, ws)
    B.moe_balance_loss_bwd(b, logits, mask, counts, grad, dl)
    return counts, prob, loss, dl, ws


def inputs(T, E, k, seed, masked):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, E, generator=g, device="cuda") * 2 + torch.randn(E, generator=g, device="cuda")
    idx = x.topk(k, 1).indices.to(torch.int32)
    mask = (torch.rand(T, generator=g, device="cuda") < 0.7).to(torch.uint8) if masked else None
    return x, idx, mask


def check(x, idx, mask, grad=None):
    counts, prob, loss, dl, ws = run(x, idx, mask, grad)
    assert B.moe_get_device_error(ws) == (0, 0)
    rc, n, rp, rl, rd = fb.balance(x.double().cpu().numpy(), idx.cpu().numpy(), ALPHA, BETA, None if mask is None else mask.cpu().numpy())
    assert np.array_equal(counts.cpu().numpy(), np.concatenate([rc, [n]]))
    tol = (x.shape[0] / 64 + 60) * 2.0 ** -23
    assert np.allclose(prob.cpu().numpy(), rp, rtol=tol, atol=1e-37)
    assert np.allclose(loss.cpu().numpy(), rl, rtol=2 * tol, atol=1e-37)
    rd = rd * (1.0 if grad is None else float(grad))
    # the size of the terms that a gradient entry is the sum of
    m, k, E = max(n, 1), idx.shape[1], x.shape[1]
    f = np.abs(E * rc / (k * m) - 1)
    lse = np.abs(np.log(np.exp(x.double().cpu().numpy()).sum(1)))
    s = torch.softmax(x.double(), 1).cpu().numpy()
    size = (ALPHA * s * (f + (s * f).sum(1, keepdims=True)) + 2 * BETA * lse[:, None] * s) / m * (1.0 if grad is None else abs(float(grad)))
    bad = np.abs(dl.double().cpu().numpy() - rd) > 2.0 ** -19 * size + 1e-37
    if mask is not None:
        bad[mask.cpu().numpy() == 0] = False
        assert not bool(dl[mask == 0].any())
    assert not bad.any()


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 2, 2), (64, 5, 3), (33, 16, 1), (1000, 64, 6), (777, 60, 4), (129, 100, 8),
                                   (50, 128, 2), (517, 129, 8), (4096, 256, 8), (31, 255, 7), (40000, 32, 2), (5, 3, 1)])
def test_against_float64(T, E, k, masked):
    check(*inputs(T, E, k, T + E, masked))


def test_upstream_gradient():
    x, idx, mask = inputs(100, 12, 2, 4, True)
    check(x, idx, mask, torch.tensor([-2.5], device="cuda"))


def test_no_token_is_left():
    x, idx, _ = inputs(40, 8, 2, 1, False)
    x[:] = float("nan")                                      # nothing of a padded token is used
    counts, prob, loss, dl, ws = run(x, idx, torch.zeros(40, dtype=torch.uint8, device="cuda"))
    for t in (counts, prob, loss, dl):
        assert not bool(t.any())


def test_masked_tokens_may_hold_anything():
    x, idx, mask = inputs(200, 24, 3, 2, True)
    ref = run(x, idx, mask)
    x[mask == 0] = float("nan")
    idx[mask == 0] = -7
    for a, b in zip(ref[:4], run(x, idx, mask)[:4]):
        assert torch.equal(a, b)


def test_experts_that_cannot_be_chosen():
    x, _, _ = inputs(60, 9, 2, 3, False)
    x[:, 4:] = float("-inf")
    check(x, x.topk(2, 1).indices.to(torch.int32), None)
    # a token with no expert at all is counted and adds nothing
    idx = x.topk(2, 1).indices.to(torch.int32)
    x[11] = float("-inf")
    counts, prob, loss, dl, _ = run(x, idx)
    assert int(counts[9]) == 60 and bool(loss.isfinite().all()) and not bool(dl[11].any()) and bool(dl.isfinite().all())
    rc, n, rp, rl, _ = fb.balance(x.double().cpu().numpy(), idx.cpu().numpy(), ALPHA, BETA)
    assert np.allclose(prob.cpu().numpy(), rp, rtol=1e-5) and np.allclose(loss.cpu().numpy(), rl, rtol=1e-5)


def test_nan_and_inf():
    x, idx, _ = inputs(60, 9, 2, 3, False)
    clean = run(x, idx)[3]
    x[7, 2], x[9, 0] = float("nan"), float("inf")
    counts, prob, loss, dl, _ = run(x, idx)
    assert int(counts.sum()) == 60 * 2 + 60 and bool(loss[0].isnan()) and bool(dl[7].isnan().all()) and not bool(dl[9].isfinite().any())
    rest = [i for i in range(60) if i not in (7, 9)]
    assert torch.equal(dl[rest], clean[rest])


def test_large_logits():
    x, idx, _ = inputs(60, 9, 2, 3, False)
    x *= 1e4
    counts, prob, loss, dl, _ = run(x, idx)
    rc, n, rp, rl, rd = fb.balance(x.double().cpu().numpy(), idx.cpu().numpy(), ALPHA, BETA)
    assert np.allclose(prob.cpu().numpy(), rp, rtol=1e-5, atol=1e-30) and np.allclose(loss.cpu().numpy(), rl, rtol=1e-5)
    assert np.allclose(dl.cpu().numpy(), rd, rtol=1e-4, atol=1e-6 * np.abs(rd).max())


def test_a_choice_that_is_no_expert():
    x, idx, _ = inputs(60, 9, 2, 3, False)
    ref = run(x, idx)[0].clone()
    lost = int(idx[5, 1])
    idx[5, 1] = 9
    counts, _, _, _, ws = run(x, idx)
    assert B.moe_get_device_error(ws)[0] == 7
    ref[lost] -= 1
    assert torch.equal(counts, ref)


def test_workspace_is_used_again_and_results_are_the_same():
    x, idx, mask = inputs(30000, 64, 6, 5, True)
    a = run(x, idx, mask)
    for _ in range(3):
        b = run(x, idx, mask, ws=a[4])
        for i in range(4):
            assert torch.equal(a[i], b[i])
    small = inputs(10, 64, 6, 6, False)
    assert torch.equal(run(*small, ws=a[4])[1], run(*small)[1])


@pytest.mark.parametrize("E,k,renorm", [(8, 2, 1), (64, 6, 1), (40, 3, 0)])
def test_router_backward_takes_it_along(E, k, renorm):
    """moe_router_bwd_aux is moe_router_bwd with the gradient added to dlogits, and dx and dw_r of that sum."""
    T, H = 200, 256
    g = torch.Generator(device="cuda").manual_seed(E)
    mk = lambda *s, std=1.0: torch.randn(*s, generator=g, device="cuda") * std  # noqa: E731
    d = B.dims(T, H, 128, E, k, renorm)
    ws = torch.zeros(B.moe_workspace_size(d, 1), dtype=torch.uint8, device="cuda")
    x, w = mk(T, H).bfloat16(), mk(E, H, std=0.05).bfloat16()
    logits = torch.zeros(T, E, device="cuda")
    B.moe_router_fwd(d, x, w, logits, ws)
    idx, prob = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    cap = B.moe_rows_capacity(d)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    B.moe_route(d, logits, idx, prob, i32(E), i32(T * k), i32(cap), torch.zeros(cap, device="cuda"), ws)
    dprob, aux, dx0 = mk(T, k, std=0.1), mk(T, E, std=0.01), mk(T, H, std=0.01).bfloat16()
    out = []
    for a in (None, aux, torch.zeros_like(aux)):
        dl, dx, dw = torch.zeros(T, E, device="cuda"), dx0.clone(), torch.zeros(E, H, device="cuda")
        B.moe_router_bwd_aux(d, x, w, logits, idx, prob, dprob, a, dl, dx, dw, ws)
        out.append((dl, dx, dw))
    dl, dx, dw = torch.zeros(T, E, device="cuda"), dx0.clone(), torch.zeros(E, H, device="cuda")
    B.moe_router_bwd(d, x, w, logits, idx, prob, dprob, dl, dx, dw, ws)
    assert torch.equal(out[0][0], dl) and torch.equal(out[0][1], dx) and torch.equal(out[0][2], dw)
    assert torch.equal(out[2][0], dl) and torch.equal(out[2][2], dw)
    total = dl.double() + aux.double()
    assert torch.allclose(out[1][0].double(), total, rtol=2.0 ** -23, atol=0)
    ref_dx = dx0.double() + total @ w.double()
    assert float((out[1][1].double() - ref_dx).abs().max()) <= 2.0 ** -8 * float(ref_dx.abs().max())
    ref_dw = total.t() @ x.double()
    # dlogits as two bf16 terms: 2^-16 of each, and float32 sums
    size = total.abs().t() @ x.double().abs()
    assert bool(((out[1][2].double() - ref_dw).abs() <= size * (2.0 ** -16 + 200 * 2.0 ** -23)).all())


def test_the_same_expert_twice():
    """A choice counts as often as it stands there."""
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(70, 6, generator=g, device="cuda")
    idx = torch.randint(0, 6, (70, 3), generator=g, device="cuda", dtype=torch.int32)
    idx[:, 2] = idx[:, 0]
    check(x, idx, None)
