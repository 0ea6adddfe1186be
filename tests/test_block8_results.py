"""What Fp8MoEBlock's results hold where nothing computes them."""
import pytest
import torch

from moe_expert_ffn_03_gb300 import build
from moe_expert_ffn_03_gb300.block8 import Fp8MoEBlock, Scratch8


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("weights", [dict(), dict(alpha=0.01, beta=0.001)])
def test_the_balance_losss_are_zeros_until_it_runs(weights, monkeypatch):
    """Without the loss (alpha = beta = 0) nothing ever writes them."""
    plain = torch.empty

    def full_of_something(*size, **kw):
        return plain(*size, **kw).fill_(77)

    scratch = Scratch8(40, 128, 256, 8, 2, device="cpu")
    monkeypatch.setattr(torch, "empty", full_of_something)
    b = Fp8MoEBlock(40, 128, 256, 8, 2, scratch=scratch, **weights)
    assert b.counts.shape == (9,) and b.counts.dtype == torch.int32 and b.prob_mean.shape == (8,)
    for t in (b.counts, b.prob_mean, b.loss):
        assert not bool(t.any())
