"""The operators around the layer take tensors of the current GPU only: a pointer into host memory, or into
another GPU's, is nothing a kernel could read."""
import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build
from moe_expert_ffn_03_gb300.block import MoEBlock

R, H, I, E = 4, 64, 64, 2
BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build.build()


def calls():
    """Name, function, and its tensor arguments (shape, type) in order, others as they are."""
    n, g, rows, wt = B.norm(R, H), B.grouped(R, H, I, E), ((R, H), BF16), ((H,), BF16)
    stat, codes, scales = ((R,), F32), ((R, H), U8), ((R, H // 32), U8)
    ws_n, ws_g = (1 << 12,), (B.moe_grouped_linear_workspace_size(g),)
    gu, a, c2, s2 = ((R, 2 * I), BF16), ((R, I), BF16), ((R, 2 * I), U8), ((R, 2 * I // 32), U8)
    ss, w = ((E,), I32), ((E, I, H), BF16)
    return {
        "layernorm_fwd": (B.moe_layernorm_fwd, [n, rows, rows, wt, wt, rows, rows, stat, stat, codes, scales]),
        "layernorm_bwd": (B.moe_layernorm_bwd, [n, rows, rows, stat, stat, None, None, wt, rows, rows, wt, wt, (ws_n, U8)]),
        "layernorm_bwd8": (B.moe_layernorm_bwd, [n, rows, None, None, stat, codes, scales, wt, rows, rows, wt, wt, (ws_n, U8)]),
        "act8_pack": (B.moe_act8_pack, [rows, codes, scales]),
        "act8_unpack": (B.moe_act8_unpack, [codes, scales, wt, wt, rows]),
        "swiglu_fwd": (B.moe_swiglu_fwd, [gu, stat, a, c2, s2]),
        "swiglu_bwd": (B.moe_swiglu_bwd, [gu, None, None, stat, a, gu, stat, a]),
        "swiglu_bwd8": (B.moe_swiglu_bwd, [None, c2, s2, stat, a, gu, stat, a]),
        "linear_fwd": (B.moe_grouped_linear_fwd, [g, rows, ss, w, a, (ws_g, U8)]),
        "linear_dgrad": (B.moe_grouped_linear_dgrad, [g, a, ss, w, rows, (ws_g, U8)]),
        "linear_wgrad": (B.moe_grouped_linear_wgrad, [g, rows, a, ss, w, (ws_g, U8)]),
    }


NAMES = ["layernorm_fwd", "layernorm_bwd", "layernorm_bwd8", "act8_pack", "act8_unpack", "swiglu_fwd", "swiglu_bwd",
         "swiglu_bwd8", "linear_fwd", "linear_dgrad", "linear_wgrad"]


def make(args, device_of):
    return [torch.zeros(*a[0], dtype=a[1], device=device_of(i)) if isinstance(a, tuple) else a for i, a in enumerate(args)]


@pytest.mark.parametrize("name", NAMES)
def test_host_tensors(name):
    f, args = calls()[name]
    with pytest.raises(ValueError, match="GPU"):
        f(*make(args, lambda i: "cpu"))


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_one_host_tensor(name):
    """Whichever of a call's tensors it is; all on the GPU, the call goes through."""
    f, args = calls()[name]
    for bad in (i for i, a in enumerate(args) if isinstance(a, tuple)):
        with pytest.raises(ValueError, match="GPU"):
            f(*make(args, lambda i: "cpu" if i == bad else "cuda"))
    f(*make(args, lambda i: "cuda"))
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_block():
    T, H, I, E, k = 8, 128, 128, 4, 2
    blk = MoEBlock(T, H, I, E, k)
    mk = lambda *s: torch.zeros(*s, dtype=BF16, device="cuda")  # noqa: E731
    w = {"gamma": mk(H), "beta": mk(H), "w_r": mk(E, H), "w_gu": mk(E, 2 * I, H), "w_d": mk(E, H, I)}
    on_host = {**w, "w_r": w["w_r"].cpu()}
    with pytest.raises(ValueError, match="GPU"):
        blk.forward(mk(T, H), on_host)
    blk.forward(mk(T, H), w)
    for dout, ww in ((mk(T, H).cpu(), w), (mk(T, H), on_host)):
        with pytest.raises(ValueError, match="GPU"):
            blk.backward(dout, ww)
    blk.backward(mk(T, H), w)
    assert blk.device_error() == (0, 0)
