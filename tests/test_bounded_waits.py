"""What a kernel's bounded waits have to keep to where they give up.

These are read off the CUDA sources: the ways in which they matter (lanes of a warp that part, memory
that goes while something is on its way) show only where a wait runs out in an unlucky moment.
"""
import ctypes
import re

from moe_expert_ffn_03_gb300 import binding as B, build
from test_pdl_waits import kernel_body, sources

# one thread only: a branch on a lane or a thread, at the call or around it
ONE_THREAD = re.compile(r"if \((?:lane|threadIdx\.x) == 0")


def wait_calls(src):
    """(line number, its text, text of the enclosing blocks' heads) of every call of a bounded wait."""
    heads, out, start = [], [], 0
    text = re.sub(r"//[^\n]*", lambda m: " " * len(m.group()), src)
    for m in re.finditer(r"[{};]|\bwait_phase(?:_\w+)?\(", text):
        if m.group() == "{":
            heads.append(text[start:m.start()])
            start = m.end()
        elif m.group() == "}":
            heads.pop()
            start = m.end()
        elif m.group() == ";":
            start = m.end()
        else:
            out.append((text.count("\n", 0, m.start()) + 1, m.group(), text[start:m.start()], list(heads)))
    return out


def test_a_warp_gives_up_together():
    """tcgen05.ld, shuffles and __syncwarp need all lanes of a warp, so a wait whose warp goes on to them
    has to end alike in all lanes; the others are a single thread's."""
    seen = 0
    for name, src in sources().items():
        for line, call, statement, heads in wait_calls(src):
            if "__device__" in statement:
                continue                                     # the definition
            seen += 1
            single = any(ONE_THREAD.search(h) for h in heads + [statement])
            assert single or call.startswith("wait_phase_warp"), f"{name}:{line}: lanes of a warp may part here"
    assert seen >= 15


def test_copies_land_after_any_wait_gave_up():
    """A producer may have issued its last copies and left when another warp's wait gives up; so it is the
    whole block, behind its last barrier, that lets copies land before its shared memory goes."""
    for file, kernel in (("grouped_linear.cu", "grouped_linear_kernel"), ("gemm.cu", "grouped_gemm_kernel")):
        body = kernel_body(sources()[file], kernel)
        end = body[body.rindex("__syncthreads();"):]
        assert re.search(r"if \((?:warp == 0 && )?\*abort_s\) \{[^}]*globaltimer_ns\(\)", end), kernel
        assert end.index("*abort_s") < end.index("cluster_sync();") < end.index("tmem_dealloc"), kernel


def test_grouped_linear_wait_selftest_checks_its_arguments():
    build.build()
    lib, P = B.lib(), ctypes.c_void_p
    A, MIS = P(256), P(260)                  # an aligned and a misaligned address; none is read
    invalid, alignment, workspace = 1, 3, 4
    g = B.grouped(40, 64, 128, 4)
    need = lib.moe_grouped_linear_workspace_size(ctypes.byref(g))

    def call(op=0, rows_in=A, other=A, ss=A, out=A, limit=20_000_000, ws=A, n_ws=need, d=g):
        return lib.moe_selftest_grouped_linear_wait(ctypes.byref(d), op, rows_in, 64, other, 128, ss, out, 0, limit, ws,
                                                    n_ws, None)

    assert call(op=3) == invalid and call(op=-1) == invalid
    assert call(limit=10) == invalid and call(limit=3 * 10 ** 9) == invalid
    for name in ("rows_in", "other", "ss", "out"):
        assert call(**{name: None}) == invalid and call(**{name: MIS}) == alignment, name
    assert call(ws=None) == workspace and call(n_ws=need - 1) == workspace
    assert call(d=B.grouped(0, 64, 128, 4)) == invalid
