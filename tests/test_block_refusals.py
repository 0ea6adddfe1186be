"""What MoEBlock refuses before anything is launched (its buffers may lie on the CPU here)."""
import pytest

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
