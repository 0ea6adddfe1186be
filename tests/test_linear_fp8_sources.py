"""What the kernels of the grouped linear layers on 8-bit operands have to keep to where they begin early and where a
wait gives up, read off the CUDA sources: it matters only in an unlucky moment."""
import os
import re

from test_pdl_waits import CSRC, kernel_body, sources

KERNELS = (("grouped_linear_fp8.cu", "grouped_linear_fp8_kernel"), ("grouped_linear_fp8_few.cu", "grouped_linear_fp8_few_kernel"))


def plain(text):
    return re.sub(r"//[^\n]*", "", text)


def test_kernels_with_a_launch_of_their_own_wait_too():
    """A launch that sets the programmatic-serialization attribute itself is found in its file: all kernels there wait."""
    files = [n for n, t in sources().items() if "cudaLaunchAttributeProgrammaticStreamSerialization" in plain(t)]
    assert {"gemm.cu", "grouped_linear.cu", "grouped_linear_fp8.cu"} <= set(files)
    text = plain(sources()["grouped_linear_fp8.cu"])
    for name in ("grouped_linear_fp8_kernel", "grouped_linear_fp8_join_kernel"):
        assert "pdl_wait();" in kernel_body(text, name), name


def test_nothing_of_earlier_kernels_is_read_before_the_wait():
    for file, kernel in KERNELS:
        body = plain(kernel_body(sources()[file], kernel))
        before, after = body.split("pdl_wait();")
        for name in ("args.split_sizes", "args.sa", "args.sb", "args.out", "args.arrived", "args.pieces", "args.plan", "l8_prefix", "l8_cut",
                     "tma_load", "f8_load", "report_error", "wait_phase"):
            assert name not in before, (kernel, name)
        assert "l8_prefix" in after
        assert before.count("{") == before.count("}") + 1, f"{kernel}: not all threads wait"
    body = plain(kernel_body(sources()["grouped_linear_fp8.cu"], "grouped_linear_fp8_join_kernel"))
    assert "a.plan" not in body.split("pdl_wait();")[0] and "a.pieces" not in body.split("pdl_wait();")[0]


def test_copies_land_after_any_wait_gave_up():
    """Behind the block's last barrier, whichever warp gave up, and before tensor memory and shared memory go."""
    for file, kernel in KERNELS:
        body = plain(kernel_body(sources()[file], kernel))
        at = body.rindex("if (warp == 0 && *abort_s) {")
        assert "__syncthreads();" in body[:at][-60:], kernel              # all warps are through
        end = body[at:]
        assert re.match(r"if \(warp == 0 && \*abort_s\) \{[^}]*globaltimer_ns\(\)", end), kernel
        together = "cluster_sync();" if "cluster_sync();" in end else "__syncthreads();"
        assert 0 < end.index(together) < end.index("dealloc"), kernel


def test_a_lane_that_has_given_up_waits_no_more():
    text = plain(open(os.path.join(CSRC, "tcgen05.cuh")).read())
    later = text[text.index("void wait_phase_warp_later("):]
    later = later[:later.index("\n}")]
    # polls counted from 256: the first that fails looks at the flag, which whoever gave up has found or left set
    assert re.search(r"if \(!wait_phase_inline\([^;]*, ok \? 1u : 256u\)\) ok = false;", later) and "__syncwarp();" in later
    wait = text[text.index("bool wait_phase_inline("):]
    wait = wait[:wait.index("\n}")]
    assert re.search(r"n = first; !mbar_try_wait\(bar, parity\); \+\+n\) \{\s*if \(\(n & 255u\) != 0\) continue;\s*if \(\*abort_flag\) return false;", wait)
    # its kernel votes before the sums go anywhere
    body = plain(kernel_body(sources()["grouped_linear_fp8.cu"], "grouped_linear_fp8_kernel"))
    last = body.rindex("wait_phase_warp_later(")
    vote = body.index("ok = __all_sync(0xFFFFFFFFu, ok);", last)
    assert all(body.index(s, last) > vote for s in ("__stcg(mine", "l8_store<MODE>(&tmO", "args.out"))


def test_waits_are_all_called():
    """Every form of a bounded wait has a caller."""
    text = plain(open(os.path.join(CSRC, "tcgen05.cuh")).read())
    names = set(re.findall(r"\b(wait_phase\w*|mbar_\w+)\([^;]*\) \{", text))
    everything = "".join(plain(t) for t in sources().values()) + "".join(
        plain(open(os.path.join(CSRC, f)).read()) for f in os.listdir(CSRC) if f.endswith(".cuh"))
    for name in sorted(names):
        assert len(re.findall(rf"\b{name}\(", everything)) >= 2, f"{name} is called nowhere"


def test_longest_tile_is_far_below_the_limit_of_the_waits():
    """The wait for a free slot of the ring of tiles lasts a tile.  A weight gradient's is the longest: its plan weighs a
    piece of one even share of the pairs, which costs two shares at most (a share and a piece), so the piece it picks
    is no longer than that; nor is any longer than all rows that fit in memory.  750 clocks a block at 2.07 GHz."""
    pairs, memory = 76, 284_208 << 20
    longest = 0.0
    for a in range(1, 200):
        for b in range(1, 200):
            K, N = 256 * (a - 1) + 16, 256 * (b - 1) + 16             # the smallest sizes with a x b tiles of 256 x 256
            blocks = min(1 << 30, memory // (K + N)) / 128
            longest = max(longest, blocks * min(1.0, 2 * a * b / pairs) * 750 / 2.07e9)
    assert 0.25 < longest < 0.32
    text = plain(sources()["grouped_linear_fp8.cu"])
    assert "fminf(ceilf(units / float(pairs)) * piece, float(share) + piece)" in text        # the plan's measure
    assert 2_000_000_000 == int(re.search(r"kWaitLimitNs = (\d+)", "".join(
        open(os.path.join(CSRC, f)).read() for f in os.listdir(CSRC)).replace("ull", "").replace("'", "")).group(1))
