"""What the operators on blocks of 128 and Fp8MoEBlock refuse before anything is launched: in the C library, in the
binding, in the block.  Nothing here needs a GPU; no address is read."""
import ctypes

import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B, build
from moe_expert_ffn_03_gb300.block8 import Fp8MoEBlock, Scratch8, Weights8

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4
A, MIS = P(256), P(260)                      # an aligned and a misaligned address
SIZES = (40, 128, 256, 8, 2)
BF16, F32, U8, I32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.fixture(scope="module")
def lib():
    return B.lib()


def changed(s, **kw):
    for k, v in kw.items():
        setattr(s, k, v)
    return ctypes.byref(s)


def test_rmsnorm(lib):
    def fwd(n=None, x=A, residual=None, gamma=A, h=None, y=A, rstd=None, codes=None, scales=None, **kw):
        return lib.moe_rmsnorm_fwd(n or changed(B.norm(4, 64), **kw), x, residual, gamma, h, y, rstd, codes, scales, None)

    assert lib.moe_rmsnorm_fwd(None, *[A] * 8, None) == INVALID
    for bad in (dict(rows=-1), dict(rows=2 ** 31 - 0), dict(H=0), dict(ld_in=63), dict(ld_out=63), dict(x_f32=2), dict(w_f32=-1),
                dict(eps=-1.0), dict(eps=float("nan"))):
        assert fwd(**bad) == INVALID, bad
    assert fwd(H=16385, ld_in=16385, ld_out=16385) == UNSUPPORTED
    assert fwd(x=None) == INVALID and fwd(gamma=None) == INVALID
    assert fwd(y=None) == INVALID                                        # nothing to write
    assert fwd(residual=A) == INVALID and fwd(h=A) == INVALID
    assert fwd(codes=A) == INVALID and fwd(scales=A) == INVALID
    for name in ("x", "gamma", "y", "rstd"):
        assert fwd(**{name: MIS}) == ALIGNMENT, name
    assert fwd(codes=MIS, scales=A) == ALIGNMENT and fwd(residual=MIS, h=A) == ALIGNMENT
    assert fwd(rows=0, x=None, y=None) == OK

    def bwd(dy=A, x=A, rstd=A, gamma=A, dres=None, dx=A, dgamma=A, ws=A, n_ws=1 << 20, **kw):
        return lib.moe_rmsnorm_bwd(changed(B.norm(4, 64), **kw), dy, x, rstd, gamma, dres, dx, dgamma, ws, n_ws, None)

    for name in ("dy", "x", "rstd", "gamma", "dx", "dgamma"):
        assert bwd(**{name: None}) == INVALID and bwd(**{name: MIS}) == ALIGNMENT, name
    assert bwd(dres=MIS) == ALIGNMENT and bwd(ws=None) == WORKSPACE and bwd(n_ws=16) == WORKSPACE and bwd(ws=P(272)) == ALIGNMENT
    assert lib.moe_rmsnorm_workspace_size(changed(B.norm(4, 64))) >= 4 * 64 * 4
    assert lib.moe_rmsnorm_workspace_size(changed(B.norm(4, 64), H=0)) == 0


def test_balance(lib):
    need = lib.moe_balance_loss_workspace_size(ctypes.byref(B.balance(8, 4, 2)))
    assert need >= 256 and lib.moe_balance_loss_workspace_size(ctypes.byref(B.balance(8, 0, 2))) == 0

    def fwd(logits=A, idx=A, mask=None, counts=A, prob=A, loss=A, ws=A, n_ws=need, T=8, E=4, k=2):
        return lib.moe_balance_loss_fwd(ctypes.byref(B.balance(T, E, k)), logits, idx, mask, counts, prob, loss, ws, n_ws, None)

    assert fwd(T=0) == INVALID and fwd(E=257) == UNSUPPORTED and fwd(E=0) == UNSUPPORTED and fwd(k=5) == UNSUPPORTED
    assert fwd(k=0) == UNSUPPORTED and fwd(T=2 ** 30, k=2) == UNSUPPORTED
    for name in ("logits", "idx", "counts", "prob", "loss"):
        assert fwd(**{name: None}) == INVALID and fwd(**{name: MIS}) == ALIGNMENT, name
    assert fwd(mask=MIS) == ALIGNMENT and fwd(ws=None) == WORKSPACE and fwd(ws=P(272)) == ALIGNMENT and fwd(n_ws=need - 1) == WORKSPACE

    def bwd(logits=A, mask=None, counts=A, grad=None, dlogits=A):
        return lib.moe_balance_loss_bwd(ctypes.byref(B.balance(8, 4, 2)), logits, mask, counts, grad, dlogits, None)

    for name in ("logits", "counts", "dlogits"):
        assert bwd(**{name: None}) == INVALID and bwd(**{name: MIS}) == ALIGNMENT, name
    assert bwd(grad=P(258)) == ALIGNMENT and bwd(mask=MIS) == ALIGNMENT


def test_block_quantizers(lib):
    def quantize(src=A, f32=0, rows=4, cols=64, ld=64, codes=A, scales=A, split=None, E=0, tc=None, ts=None, fmt=1):
        return lib.moe_fp8_block_quantize(src, f32, rows, cols, ld, codes, scales, split, E, tc, ts, fmt, None)

    assert quantize(rows=-1) == INVALID and quantize(cols=0, ld=0) == INVALID and quantize(ld=63) == INVALID and quantize(f32=2) == INVALID
    assert quantize(codes=None) == INVALID and quantize(scales=None) == INVALID and quantize(codes=None, scales=None) == INVALID
    assert quantize(tc=A, ts=A) == INVALID                               # no sizes of the experts
    assert quantize(tc=A, split=A, E=2) == INVALID and quantize(tc=A, ts=A, split=A, E=2, fmt=0) == INVALID
    assert quantize(split=A, E=0) == UNSUPPORTED and quantize(split=A, E=257) == UNSUPPORTED
    assert quantize(src=None) == INVALID and quantize(src=MIS) == ALIGNMENT and quantize(codes=MIS) == ALIGNMENT
    assert quantize(tc=A, ts=MIS, split=A, E=2) == ALIGNMENT and quantize(rows=0, src=None) == OK

    def weights(w=A, f32=0, E=1, N=64, K=64, codes=A, scales=A):
        return lib.moe_fp8_block_quantize_weights(w, f32, E, N, K, codes, scales, None)

    for name in ("w", "codes", "scales"):
        assert weights(**{name: None}) == INVALID and weights(**{name: MIS}) == ALIGNMENT, name
    assert weights(E=0) == INVALID and weights(K=0) == INVALID and weights(N=2 ** 21) == UNSUPPORTED and weights(f32=-1) == INVALID

    def back(codes=A, scales=A, fmt=0, rows=256, mat=0, cols=64, dst=A, f32=0, ld=64):
        return lib.moe_fp8_block_dequantize(codes, scales, fmt, rows, mat, cols, dst, f32, ld, None)

    for name in ("codes", "scales", "dst"):
        assert back(**{name: None}) == INVALID and back(**{name: MIS}) == ALIGNMENT, name
    assert back(fmt=3) == INVALID and back(fmt=-1) == INVALID and back(ld=63) == INVALID and back(f32=2) == INVALID
    assert back(mat=100, fmt=2) == INVALID and back(mat=128, fmt=0) == INVALID and back(mat=-1) == INVALID

    def pack(T=4, k=2, E=8, cols=64, ws=A, **kw):
        p = dict(codes=A, scales=A, idx=A, prob=A, row_of=A, split=A)
        o = dict(codes_out=A, scales_out=A, prob_rows=A, pos_of=A)
        p.update({n: v for n, v in kw.items() if n in p})
        o.update({n: v for n, v in kw.items() if n in o})
        return lib.moe_fp8_block_pack(*p.values(), T, k, E, cols, *o.values(), ws, None)

    for name in ("codes", "scales", "idx", "prob", "row_of", "split", "codes_out", "scales_out", "prob_rows", "pos_of"):
        assert pack(**{name: None}) == INVALID and pack(**{name: MIS}) == ALIGNMENT, name
    assert pack(T=-1) == INVALID and pack(k=9) == UNSUPPORTED and pack(k=0) == UNSUPPORTED and pack(E=1) == UNSUPPORTED
    assert pack(cols=40) == UNSUPPORTED and pack(ws=None) == WORKSPACE and pack(ws=P(272)) == ALIGNMENT and pack(E=257) == UNSUPPORTED


def test_grouped_linear(lib):
    g = B.grouped(4, 64, 128, 2)
    need = lib.moe_grouped_linear_fp8_workspace_size(ctypes.byref(g))
    assert need >= 256
    for K, N in ((8, 64), (64, 8), (72, 64), (64, 24)):
        bad = ctypes.byref(B.grouped(4, K, N, 2))
        assert lib.moe_grouped_linear_fp8_workspace_size(bad) == 0
        assert lib.moe_grouped_linear_fp8_fwd(bad, A, A, A, A, A, A, 128, A, need, None) == UNSUPPORTED
    names = ("a", "sa", "ss", "b", "sb", "out")

    def call(f, ld=128, ws=A, n_ws=need, d=g, **kw):
        p = {**dict.fromkeys(names, A), **kw}
        return f(ctypes.byref(d), *[p[n] for n in names], ld, ws, n_ws, None)

    def wgrad(ws=A, n_ws=need, d=g, **kw):
        order = ("a", "sa", "b", "sb", "ss", "out")
        p = {**dict.fromkeys(names, A), **kw}
        return lib.moe_grouped_linear_fp8_wgrad(ctypes.byref(d), *[p[n] for n in order], ws, n_ws, None)

    fwd, dgrad = lib.moe_grouped_linear_fp8_fwd, lib.moe_grouped_linear_fp8_dgrad
    for c in (lambda **kw: call(fwd, **kw), lambda **kw: call(dgrad, **kw), wgrad):
        for name in names:
            assert c(**{name: None}) == INVALID and c(**{name: MIS}) == ALIGNMENT, name
        assert c(ws=None) == WORKSPACE and c(n_ws=need - 1) == WORKSPACE and c(ws=P(272)) == ALIGNMENT
        assert c(d=B.grouped(-1, 64, 128, 2)) == INVALID and c(d=B.grouped(4, 64, 128, 257)) == UNSUPPORTED
    assert call(fwd, ld=127) == INVALID and call(fwd, ld=132) == UNSUPPORTED and call(dgrad, ld=63) == INVALID
    assert lib.moe_grouped_linear_fp8_fwd(None, *[A] * 6, 128, A, need, None) == INVALID
    assert call(fwd, d=B.grouped(0, 64, 128, 2), a=None) == OK

    def wait(op=0, limit=20_000_000, d=g, **kw):
        p = {**dict.fromkeys(("a", "sa", "b", "sb", "ss", "out"), A), **kw}
        return lib.moe_selftest_grouped_linear_fp8_wait(ctypes.byref(d), op, *p.values(), 0, limit, A, need, None)

    assert wait(op=3) == INVALID and wait(op=-1) == INVALID and wait(limit=10) == INVALID and wait(limit=3 * 10 ** 9) == INVALID
    assert wait(a=None) == INVALID and wait(out=MIS) == ALIGNMENT and wait(d=B.grouped(0, 64, 128, 2)) == INVALID


def test_router_backward_with_a_gradient(lib):
    d = B.dims(4, 128, 128, 4, 2)
    assert lib.moe_router_bwd_aux(ctypes.byref(d), *[A] * 6, MIS, *[A] * 4, 1 << 30, None) == ALIGNMENT


# ---- binding: types, shapes, devices ---------------------------------------------------------------
def new(*s, dt=BF16):
    return torch.zeros(*s, dtype=dt)


def calls():
    """Name, function, its arguments: tensors all on the CPU, right otherwise."""
    R, H, N, E, k = 4, 64, 128, 2, 2
    n, g, b, nb = B.norm(R, H), B.grouped(R, H, N, E), B.balance(R, E, k), B.fp8_blocks(R, E)
    ws = new(B.moe_grouped_linear_fp8_workspace_size(g), dt=U8)
    x8, xs, dy8, dys = new(R, H, dt=U8), new(1, R, dt=F32), new(R, N, dt=U8), new(1, R, dt=F32)
    w8, w8s, ss = new(E, N, H, dt=U8), new(E, 1, 1, dt=F32), new(E, dt=I32)
    xt, xts, dyt, dyts = new(nb * 128, H, dt=U8), new(nb, 1, dt=F32), new(nb * 128, N, dt=U8), new(nb, N, dt=F32)
    ik, pk, T = new(R, k, dt=I32), new(R, k, dt=F32), R
    return {
        "rmsnorm_fwd": (B.moe_rmsnorm_fwd, [n, new(R, H), new(R, H), new(H), new(R, H), new(R, H), new(R, dt=F32), x8, xs]),
        "rmsnorm_bwd": (B.moe_rmsnorm_bwd, [n, new(R, H), new(R, H), new(R, dt=F32), new(H), new(R, H), new(R, H), new(H), new(4096, dt=U8)]),
        "balance_fwd": (B.moe_balance_loss_fwd, [b, new(T, E, dt=F32), ik, new(T, dt=U8), new(E + 1, dt=I32), new(E, dt=F32), new(3, dt=F32),
                                                 new(B.moe_balance_loss_workspace_size(b), dt=U8)]),
        "balance_bwd": (B.moe_balance_loss_bwd, [b, new(T, E, dt=F32), new(T, dt=U8), new(E + 1, dt=I32), new(1, dt=F32), new(T, E, dt=F32)]),
        "quantize": (B.moe_fp8_block_quantize, [new(R, H), x8, xs, ss, xt, new(nb, H, dt=F32)]),
        "quantize_weights": (B.moe_fp8_block_quantize_weights, [new(E, N, H), w8, w8s]),
        "dequantize": (B.moe_fp8_block_dequantize, [x8, xs, "rows", new(R, H)]),
        "dequantize_weights": (B.moe_fp8_block_dequantize, [w8, w8s, "tiles", new(E, N, H)]),
        "pack": (B.moe_fp8_block_pack, [x8, xs, ik, pk, new(R, k, dt=I32), ss, new(R * k, H, dt=U8), new(1, R * k, dt=F32),
                                        new(R * k, dt=F32), new(R, k, dt=I32), new(256, dt=U8)]),
        "linear_fwd": (B.moe_grouped_linear_fp8_fwd, [g, x8, xs, ss, w8, w8s, new(R, N), ws]),
        "linear_dgrad": (B.moe_grouped_linear_fp8_dgrad, [g, dy8, dys, ss, w8, w8s, new(R, H), ws]),
        "linear_wgrad": (B.moe_grouped_linear_fp8_wgrad, [g, xt, xts, dyt, dyts, ss, new(E, N, H), ws]),
    }


NAMES = ["rmsnorm_fwd", "rmsnorm_bwd", "balance_fwd", "balance_bwd", "quantize", "quantize_weights", "dequantize",
         "dequantize_weights", "pack", "linear_fwd", "linear_dgrad", "linear_wgrad"]


@pytest.mark.parametrize("name", NAMES)
def test_host_tensors(name):
    f, args = calls()[name]
    with pytest.raises(ValueError, match="GPU"):
        f(*args)


@pytest.mark.parametrize("name", NAMES)
def test_types_and_sizes(name):
    """A tensor of another type, or with less in it than the call would read or write."""
    f, args = calls()[name]
    for i, t in enumerate(args):
        if not isinstance(t, torch.Tensor) or t.numel() >= 4096 and t.dtype == U8 and t.dim() == 1:
            continue                                         # workspaces: the library looks at their sizes
        other = {BF16: torch.float16, F32: torch.float64, U8: torch.int8, I32: torch.int64}[t.dtype]
        for bad in (t.to(other), t.flatten()[:-1] if t.dim() == 1 else t[:-1]):
            if name in ("quantize", "quantize_weights", "dequantize", "dequantize_weights", "pack") and i == 0 and bad.dtype == t.dtype:
                continue                                     # the sizes are this tensor's
            changed_args = list(args)
            changed_args[i] = bad
            with pytest.raises((ValueError, B.MoeError)):
                f(*changed_args)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_one_host_tensor(name):
    """Whichever of a call's tensors it is; all on the GPU, the call goes through."""
    f, args = calls()[name]
    on_gpu = [a.cuda() if isinstance(a, torch.Tensor) else a for a in args]
    for i, a in enumerate(args):
        if isinstance(a, torch.Tensor):
            with pytest.raises(ValueError, match="GPU"):
                f(*on_gpu[:i], a, *on_gpu[i + 1:])
    f(*on_gpu)
    torch.cuda.synchronize()


def test_shapes_of_values_back():
    with pytest.raises(ValueError, match="blocks"):
        B.moe_fp8_block_dequantize(new(100, 64, dt=U8), new(1, 64, dt=F32), "tokens", new(100, 64))
    with pytest.raises(ValueError, match="shape"):
        B.moe_fp8_block_dequantize(new(2, 64, 64, dt=U8), new(2, 1, 1, dt=F32), "tiles", new(2, 64, 32))
    with pytest.raises(KeyError):
        B.moe_fp8_block_dequantize(new(128, 64, dt=U8), new(1, 64, dt=F32), "columns", new(128, 64))


# ---- block ---------------------------------------------------------------------------------------
def weights(T, H, I, E, k, **other):
    w = {"gamma": new(H), "w_r": new(E, H), "w_gu": Weights8(E, 2 * I, H, device="cpu"), "w_d": Weights8(E, H, I, device="cpu")}
    return {**w, **other}


@pytest.mark.parametrize("place,value", [(0, 80), (0, 20), (1, 256), (2, 128), (3, 16), (4, 1)])
def test_scratch_of_other_sizes(place, value):
    other = list(SIZES)
    other[place] = value
    with pytest.raises(ValueError, match="scratch"):
        Fp8MoEBlock(*SIZES, scratch=Scratch8(*other, device="cpu"))


def test_scratch_for_inference():
    s = Scratch8(*SIZES, device="cpu", training=False)
    with pytest.raises(ValueError, match="inference"):
        Fp8MoEBlock(*SIZES, scratch=s)
    assert Fp8MoEBlock(*SIZES, scratch=s, training=False).s is s


T, H = SIZES[:2]
BAD_ROWS = {"short": lambda: new(T - 1, H), "narrow": lambda: new(T, H // 2), "float32": lambda: new(T, H, dt=F32),
            "expanded": lambda: new(1, 1).expand(T, H), "one row for all": lambda: new(1, H).expand(T, H),
            "transposed": lambda: new(H, T).t(), "pitched": lambda: new(T, H + 8)[:, :H], "on the host": lambda: new(T, H)}


@pytest.mark.parametrize("kind", BAD_ROWS)
@pytest.mark.parametrize("which", ["x", "residual", "dout"])
def test_rows_that_would_be_read_past_their_end(which, kind):
    blk, bad = Fp8MoEBlock(*SIZES, device="cpu"), BAD_ROWS[kind]()
    with pytest.raises(ValueError):
        if which == "dout":
            blk.backward(bad, weights(*SIZES))
        else:
            blk.forward(bad if which == "x" else new(T, H), weights(*SIZES), bad if which == "residual" else None)


def test_weights_of_other_shapes():
    E, I = SIZES[3], SIZES[2]
    with pytest.raises(ValueError, match="shape"):
        Weights8(E, 2 * I, H, device="cpu").quantize(new(E, 2 * I, H // 2))
    for other in (dict(w_r=new(E - 1, H)), dict(w_gu=Weights8(E, I, H, device="cpu")), dict(w_d=Weights8(E, H, 2 * I, device="cpu"))):
        blk = Fp8MoEBlock(*SIZES, device="cpu")
        with pytest.raises(ValueError):
            blk.forward(new(T, H), weights(*SIZES, **other))
