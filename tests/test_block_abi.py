"""Host-side refusals of the operators around the layer, in the C library and in the binding:
they answer before anything is launched and need no GPU."""
import ctypes

import pytest
import torch

from moe_expert_ffn_03_gb300 import binding as B
from moe_expert_ffn_03_gb300 import build

P, I64 = ctypes.c_void_p, ctypes.c_int64
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, 1, 2, 3, 4
A, MIS = P(256), P(260)                      # an aligned and a misaligned address; none is read


@pytest.fixture(scope="module")
def lib():
    build.build()
    return B.lib()


def norm(**kw):
    n = B.norm(4, 64)
    for k, v in kw.items():
        setattr(n, k, v)
    return ctypes.byref(n)


def fwd(lib, n, x=A, residual=None, gamma=A, beta=A, h=None, y=A, mean=None, rstd=None, codes=None, scales=None):
    return lib.moe_layernorm_fwd(n, x, residual, gamma, beta, h, y, mean, rstd, codes, scales, None)


def test_layernorm_forward(lib):
    assert lib.moe_layernorm_fwd(None, *[A] * 10, None) == INVALID
    for bad in (dict(rows=-1), dict(rows=2 ** 31), dict(H=0), dict(ld_in=63), dict(ld_out=63), dict(x_f32=2),
                dict(w_f32=-1), dict(eps=-1.0), dict(eps=float("nan"))):
        assert fwd(lib, norm(**bad)) == INVALID, bad
    assert fwd(lib, norm(H=16385, ld_in=16385, ld_out=16385)) == UNSUPPORTED
    assert fwd(lib, norm(), x=None) == INVALID and b"x is NULL" in lib.moe_last_error_message()
    assert fwd(lib, norm(), gamma=None) == INVALID and fwd(lib, norm(), y=None) == INVALID
    assert fwd(lib, norm(), residual=A) == INVALID                       # no place for the sum
    assert fwd(lib, norm(), h=A) == INVALID
    assert fwd(lib, norm(), codes=A) == INVALID and fwd(lib, norm(), scales=A) == INVALID
    for name in ("x", "gamma", "beta", "y", "mean", "rstd"):
        assert fwd(lib, norm(), **{name: MIS}) == ALIGNMENT, name
    assert fwd(lib, norm(), codes=MIS, scales=A) == ALIGNMENT
    assert fwd(lib, norm(rows=0), x=None, y=None) == OK                  # nothing to do


def bwd(lib, n, dy=A, x=A, mean=A, rstd=A, codes=None, scales=None, gamma=A, dres=None, dx=A, dgamma=A, dbeta=A, ws=A,
        n_ws=1 << 20):
    return lib.moe_layernorm_bwd(n, dy, x, mean, rstd, codes, scales, gamma, dres, dx, dgamma, dbeta, ws, n_ws, None)


def test_layernorm_backward(lib):
    assert bwd(lib, norm(), x=None, mean=None) == INVALID                # neither source of n
    assert bwd(lib, norm(), codes=A, scales=A) == INVALID                # both
    assert bwd(lib, norm(), mean=None) == INVALID and bwd(lib, norm(), codes=A) == INVALID
    for name in ("dy", "rstd", "gamma", "dx", "dgamma"):
        assert bwd(lib, norm(), **{name: None}) == INVALID, name
        assert bwd(lib, norm(), **{name: MIS}) == ALIGNMENT, name
    assert bwd(lib, norm(), dres=MIS) == ALIGNMENT and bwd(lib, norm(), dbeta=MIS) == ALIGNMENT
    assert bwd(lib, norm(), ws=None) == WORKSPACE and bwd(lib, norm(), n_ws=16) == WORKSPACE
    assert bwd(lib, norm(), ws=P(272)) == ALIGNMENT
    assert lib.moe_layernorm_workspace_size(norm()) >= 4 * 2 * 64 * 4
    assert lib.moe_layernorm_workspace_size(norm(H=0)) == 0


def test_act8(lib):
    pack = lambda src=A, rows=4, cols=64, ld=64, codes=A, scales=A: lib.moe_act8_pack(  # noqa: E731
        src, 0, rows, cols, ld, codes, scales, None)
    assert pack(rows=-1) == INVALID and pack(cols=0) == INVALID and pack(ld=63) == INVALID
    assert pack(src=None) == INVALID and pack(codes=None) == INVALID and pack(scales=MIS) == ALIGNMENT
    assert pack(rows=0, src=None) == OK
    unpack = lambda gamma=None, beta=None, cols=64, ld=64, rows=4, dst=A: lib.moe_act8_unpack(  # noqa: E731
        A, A, rows, cols, gamma, beta, 0, dst, 0, ld, None)
    assert unpack(beta=A) == INVALID and unpack(gamma=MIS) == ALIGNMENT and unpack(dst=None) == INVALID
    assert unpack(ld=1) == INVALID and unpack(rows=0, dst=None) == OK


def test_swiglu(lib):
    f = lambda rows=4, I=64, gu=A, ld_gu=128, a=A, ld_a=64, prob=None, codes=None, scales=None: lib.moe_swiglu_fwd(  # noqa: E731
        rows, I, gu, ld_gu, prob, a, ld_a, codes, scales, None)
    assert f(I=0) == INVALID and f(ld_gu=127) == INVALID and f(ld_a=63) == INVALID and f(rows=-5) == INVALID
    assert f(gu=None) == INVALID and f(a=MIS) == ALIGNMENT and f(prob=MIS) == ALIGNMENT
    assert f(codes=A) == INVALID and f(rows=0, gu=None) == OK
    b = lambda rows=4, gu=A, ld_gu=128, codes=None, scales=None, prob=A, da=A, ld_da=64, dgu=A, ld_dgu=128, dprob=A,  \
        a=None, ld_a=0: lib.moe_swiglu_bwd(rows, 64, gu, ld_gu, codes, scales, prob, da, ld_da, dgu, ld_dgu, dprob, a, ld_a, None)  # noqa: E731
    assert b(gu=None) == INVALID and b(codes=A, scales=A) == INVALID     # neither, both
    assert b(prob=None) == INVALID                                       # dprob of nothing
    assert b(a=A, ld_a=63) == INVALID and b(ld_dgu=127) == INVALID and b(ld_da=1) == INVALID
    assert b(da=None) == INVALID and b(dgu=MIS) == ALIGNMENT and b(dprob=MIS) == ALIGNMENT
    assert b(rows=0, gu=None) == OK


def test_grouped_linear(lib):
    g = B.grouped(40, 64, 128, 4)
    need = lib.moe_grouped_linear_workspace_size(ctypes.byref(g))
    assert need >= 256

    def f(ldx=64, ldy=128, x=A, ss=A, w=A, y=A, ws=A, n_ws=need, **kw):
        d = B.grouped(40, 64, 128, 4)
        for k, v in kw.items():
            setattr(d, k, v)
        return lib.moe_grouped_linear_fwd(ctypes.byref(d), x, ldx, ss, w, y, ldy, ws, n_ws, None)

    assert f(rows=-1) == INVALID and f(rows=2 ** 30 + 1) == INVALID
    assert f(K=60) == UNSUPPORTED and f(N=0) == UNSUPPORTED and f(E=257) == UNSUPPORTED and f(E=0) == UNSUPPORTED
    assert f(ldx=56) == INVALID and f(ldx=68) == UNSUPPORTED and f(ldy=130) == UNSUPPORTED
    for name in ("x", "ss", "w", "y"):
        assert f(**{name: None}) == INVALID, name
        assert f(**{name: MIS}) == ALIGNMENT, name
    assert f(ws=None) == WORKSPACE and f(n_ws=need - 1) == WORKSPACE and f(ws=P(272)) == ALIGNMENT
    assert f(rows=0, x=None, y=None) == OK
    d = ctypes.byref(g)
    assert lib.moe_grouped_linear_dgrad(d, None, 128, A, A, A, 64, A, need, None) == INVALID
    assert lib.moe_grouped_linear_wgrad(d, A, 64, A, 128, A, None, A, need, None) == INVALID
    assert lib.moe_grouped_linear_workspace_size(ctypes.byref(B.grouped(4, 60, 64, 1))) == 0


def test_binding_checks_types_and_shapes():
    """What would make a kernel read past a tensor's end is refused in Python."""
    b16 = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    n = B.norm(4, 64)
    for x, y, gamma in ((b16(3, 64), b16(4, 64), b16(64)), (b16(4, 64).float(), b16(4, 64), b16(64)),
                        (b16(4, 64), b16(4, 72)[:, :64], b16(64)), (b16(4, 64), b16(4, 64), b16(32)),
                        (b16(4, 64), b16(4, 64), b16(64).float()), (b16(64, 4).t(), b16(4, 64), b16(64))):
        with pytest.raises(ValueError):
            B.moe_layernorm_fwd(n, x, None, gamma, None, None, y, None, None)
    with pytest.raises(ValueError):
        B.moe_layernorm_fwd(n, b16(4, 64), None, b16(64), None, None, b16(4, 64), None, None, u8(4, 64), u8(4, 1))
    with pytest.raises(ValueError):
        B.moe_act8_pack(b16(4, 64).half(), u8(4, 64), u8(4, 2))
    with pytest.raises(ValueError):
        B.moe_act8_unpack(u8(4, 64), u8(4, 2), None, None, b16(3, 64))
    with pytest.raises(ValueError):
        B.moe_swiglu_fwd(b16(4, 100), None, b16(4, 64))
    with pytest.raises(ValueError):
        B.moe_swiglu_bwd(None, u8(4, 128), u8(4, 3), None, b16(4, 64), b16(4, 128))
    g = B.grouped(40, 64, 128, 4)
    ss = torch.zeros(4, dtype=torch.int32)
    for x, w, split in ((b16(39, 64), b16(4, 128, 64), ss), (b16(40, 64), b16(3, 128, 64), ss),
                        (b16(40, 64), b16(4, 128, 64), ss.long()), (b16(40, 64), b16(4, 64, 128).transpose(1, 2), ss)):
        with pytest.raises(ValueError):
            B.moe_grouped_linear_fwd(g, x, split, w, b16(40, 128), u8(1024))


def test_grouped_linear_kernel_waits_before_it_reads():
    """It is launched with programmatic stream serialization: everything that reads another kernel's
    output comes after pdl_wait()."""
    from test_pdl_waits import kernel_body, sources
    src = sources()["grouped_linear.cu"]
    assert "cudaLaunchAttributeProgrammaticStreamSerialization" in src
    body = kernel_body(src, "grouped_linear_kernel")
    wait = body.index("pdl_wait();")
    for access in ("args.split_sizes", "tma_load_", "args.out"):
        assert wait < body.index(access), access
