"""The grouped linear kernel's bounded waits: they run out when nothing moves, and only then.

No case here faults: producers that issue no loads leave every wait without its phase, and each gives up
at the limit and records it."""
import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build

pytestmark = pytest.mark.gpu
TIMEOUT = 6                                  # MOE_ERR_DEVICE_TIMEOUT
CALLS = (B.moe_grouped_linear_fwd, B.moe_grouped_linear_dgrad, B.moe_grouped_linear_wgrad)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    yield
    torch.cuda.empty_cache()


def ones(*s):
    return torch.ones(*s, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("op", [0, 1, 2])
@pytest.mark.parametrize("split,K,N", [([40, 0, 9, 128], 136, 264), ([2, 1], 2048, 1024)], ids=["tiles", "cut tiles"])
def test_waits_run_out_and_the_next_call_is_right(op, split, K, N):
    """As the header says, the workspace is zero-filled before its next use: calls that cut tiles leave counts."""
    R, E = sum(split), len(split)
    g = B.grouped(R, K, N, E)
    ss = torch.tensor(split, dtype=torch.int32, device="cuda")
    ws = torch.zeros(B.moe_grouped_linear_workspace_size(g), dtype=torch.uint8, device="cuda")
    x, dy, w, dw = ones(R, K), ones(R, N), ones(E, N, K), ones(E, N, K)
    rows_in, other, out = ((x, w, dy.clone()), (dy, w, x.clone()), (x, dy, dw))[op]
    B.moe_selftest_grouped_linear_wait(g, op, rows_in, other, ss, out, ws, loads=False, limit_ns=20_000_000)
    code, site = B.moe_get_device_error(ws)
    assert code == TIMEOUT and 700 <= site < 710, (code, site)
    ws.zero_()
    out.fill_(77)
    if op == 2:
        CALLS[op](g, rows_in, other, ss, out, ws)
        want = ss.view(E, 1, 1).expand(E, N, K)
    else:
        CALLS[op](g, rows_in, ss, w, out, ws)
        want = torch.full(out.shape, (K, N)[op], device="cuda")
    assert B.moe_get_device_error(ws) == (0, 0)
    assert torch.equal(out.float(), want.bfloat16().float())


def test_a_long_contraction_is_no_timeout():
    """76 experts of 2^21 rows (a multiple of 16: nothing to clear) and 84 of 17 behind them: the epilogue
    waits through 32768 steps for its accumulator, and the warp that clears rows past an expert's end
    through a whole such tile for its first.  Both take several times the limit while stages go by."""
    split = [2 ** 21] * 76 + [17] * 84
    R, E = sum(split), len(split)
    g = B.grouped(R, 8, 8, E)
    ss = torch.tensor(split, dtype=torch.int32, device="cuda")
    ws = torch.zeros(B.moe_grouped_linear_workspace_size(g), dtype=torch.uint8, device="cuda")
    x, dy, dw = ones(R, 8), ones(R, 8), torch.full((E, 8, 8), 77, dtype=torch.bfloat16, device="cuda")
    limit_ms = 1
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    B.moe_selftest_grouped_linear_wait(g, 2, x, dy, ss, dw, ws, loads=True, limit_ns=limit_ms * 1_000_000)
    b.record()
    b.synchronize()
    assert B.moe_get_device_error(ws) == (0, 0)
    assert torch.equal(dw.float(), ss.view(E, 1, 1).expand(E, 8, 8).float())     # powers of two and 17: exact
    assert a.elapsed_time(b) > 4 * limit_ms, "the call is too short to show anything"
