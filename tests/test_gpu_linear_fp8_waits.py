"""The bounded waits of the grouped linear kernels on 8-bit operands: they run out when nothing moves.

No case here faults: producers that issue no loads leave every wait without its phase, and each gives up at the
limit and records it."""
import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build

pytestmark = pytest.mark.gpu
TIMEOUT = 6                                  # MOE_ERR_DEVICE_TIMEOUT
ONE = 0x38                                   # E4M3's 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()
    yield
    torch.cuda.empty_cache()


def codes(*s):
    return torch.full(s, ONE, dtype=torch.uint8, device="cuda")


def ones(*s):
    return torch.ones(*s, device="cuda")


@pytest.mark.parametrize("op", [0, 1, 2])
@pytest.mark.parametrize("split,K,N", [([400, 0, 90, 1280], 272, 528), ([2, 1], 2048, 1024)], ids=["tiles", "few rows"])
def test_waits_run_out_and_the_next_call_is_right(op, split, K, N):
    """As the header says, the workspace is zero-filled before its next use: calls that cut tiles leave counts."""
    R, E = sum(split), len(split)
    cut = lambda n: -(-n // 128)  # noqa: E731
    g, nb = B.grouped(R, K, N, E), B.fp8_blocks(R, E)
    ss = torch.tensor(split, dtype=torch.int32, device="cuda")
    ws = torch.zeros(B.moe_grouped_linear_fp8_workspace_size(g), dtype=torch.uint8, device="cuda")
    if op == 2:
        a, sa, b, sb = torch.zeros(nb * 128, N, dtype=torch.uint8, device="cuda"), ones(nb, N), codes(nb * 128, K), ones(nb, cut(K))
        at = 0
        for n in split:
            a[at: at + n] = ONE
            at += cut(n) * 128
    else:
        c = (K, N)[op]
        a, sa, b, sb = codes(R, c), ones(cut(c), R), codes(E, N, K), ones(E, cut(N), cut(K))
    out = torch.full((R, (N, K)[op]) if op < 2 else (E, N, K), 77.0, dtype=torch.bfloat16, device="cuda")
    B.moe_selftest_grouped_linear_fp8_wait(g, op, a, sa, b, sb, ss, out, ws, loads=False, limit_ns=20_000_000)
    code, site = B.moe_get_device_error(ws)
    assert code == TIMEOUT and 720 <= site < 730, (code, site)
    ws.zero_()
    B.moe_selftest_grouped_linear_fp8_wait(g, op, a, sa, b, sb, ss, out, ws, loads=True, limit_ns=2_000_000_000)
    assert B.moe_get_device_error(ws) == (0, 0)
    want = ss.view(E, 1, 1).expand(E, N, K) if op == 2 else torch.full(out.shape, (K, N)[op], device="cuda")
    assert torch.equal(out.float(), want.bfloat16().float())
