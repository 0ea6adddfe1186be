"""What MoEBlock refuses before anything is launched (its buffers may lie on the CPU here)."""
import pytest
import torch

from moe_expert_ffn_03_gb300 import build
from moe_expert_ffn_03_gb300.block import MoEBlock, Scratch

SIZES = (40, 128, 256, 8, 2)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


@pytest.mark.parametrize("place,value", [(0, 80), (0, 20), (1, 256), (2, 128), (3, 16), (4, 1)])
def test_scratch_of_other_sizes(place, value):
    """All calls take their sizes from the scratch; the block's own tensors have the block's."""
    other = list(SIZES)
    other[place] = value
    with pytest.raises(ValueError, match="scratch"):
        MoEBlock(*SIZES, scratch=Scratch(*other, device="cpu"))


def test_scratch_of_the_same_sizes():
    s = Scratch(*SIZES, device="cpu")
    assert MoEBlock(*SIZES, scratch=s).s is s


def made(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def weights(T, H, I, E, k, **other):
    w = {"gamma": made(H), "beta": made(H), "w_r": made(E, H), "w_gu": made(E, 2 * I, H), "w_d": made(E, H, I)}
    return {**w, **other}


T, H = SIZES[:2]
BAD_ROWS = {"short": lambda: made(T - 1, H), "narrow": lambda: made(T, H // 2), "float32": lambda: made(T, H, dtype=torch.float32),
            "expanded": lambda: made(1, 1).expand(T, H), "one row for all": lambda: made(1, H).expand(T, H),
            "transposed": lambda: made(H, T).t(), "pitched": lambda: made(T, H + 8)[:, :H]}


@pytest.mark.parametrize("kind", BAD_ROWS)
@pytest.mark.parametrize("which", ["x", "residual", "dout"])
def test_rows_that_would_be_read_past_their_end(which, kind):
    """The gradient that reaches the block may be expanded from one value; the packing's call would read T * H
    values behind its pointer."""
    blk, bad = MoEBlock(*SIZES, device="cpu"), BAD_ROWS[kind]()
    with pytest.raises(ValueError):
        if which == "dout":
            blk.backward(bad, weights(*SIZES))
        else:
            blk.forward(bad if which == "x" else made(T, H), weights(*SIZES), bad if which == "residual" else None)


@pytest.mark.parametrize("w_r", [made(7, 128), made(8, 64), made(8, 128, dtype=torch.float32), made(128, 8).t()],
                         ids=["few experts", "narrow", "float32", "transposed"])
def test_router_weights(w_r):
    blk = MoEBlock(*SIZES, device="cpu")
    with pytest.raises(ValueError):
        blk.forward(made(T, H), weights(*SIZES, w_r=w_r))
    with pytest.raises(ValueError):
        blk.backward(made(T, H), weights(*SIZES, w_r=w_r))


def test_backward_before_forward():
    """The places of the rows would be whatever the memory held, and rows would be written there."""
    blk = MoEBlock(*SIZES, device="cpu")
    with pytest.raises(RuntimeError, match="before forward"):
        blk.backward(made(T, H), weights(*SIZES))
