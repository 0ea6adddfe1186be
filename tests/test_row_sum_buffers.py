"""The sums over a row's threads: two in a row use different buffers.

row_sum has one barrier, between the warps' writes and their reads.  A warp that is done reading may write the
next sum's share while another still reads, so the next sum goes to another buffer; the one after may use the
first again, since its writers have passed the barrier between.  What goes wrong otherwise (warps with different
sums, which then part at the next barrier) shows only where one warp is late, so it is read off the CUDA sources.
"""
import re

from test_pdl_waits import sources


def code(name):
    return re.sub(r"//[^\n]*", "", sources()[name])


def calls(text):
    """(buffer, position behind the statement) of every call of row_sum."""
    return [(m.group(1).strip(), m.end()) for m in re.finditer(r"\brow_sum<\d+>\([^;]*,\s*([^,;]+)\);", text)]


def test_every_user_is_looked_at():
    assert {n for n in sources() if "row_sum<" in code(n)} == {"act8.cu", "norm.cu", "rmsnorm.cu"}
    assert len(calls(code("act8.cu"))) == 1                      # one sum in a thread's life: a row each


def test_root_mean_square_norm_takes_turns():
    """All sums are in sums[flip], and flip changes behind each: at once, or in the head of the loop around it."""
    text = code("rmsnorm.cu")
    found = calls(text)
    assert len(found) == 3
    for buffer, end in found:
        assert buffer == "sums[flip]", buffer
        at_once = re.match(r"\s*flip \^= 1;", text[end:])
        heads = [m for m in re.finditer(r"for \([^{]*flip \^= 1\) \{", text[:end])]
        in_loop = heads and text.count("{", heads[-1].start(), end) > text.count("}", heads[-1].start(), end)
        assert at_once or in_loop, text[end - 200:end]
    # the second loop goes on where the first has stopped
    assert "rms_fwd_rescaled<T, VEC, NV>(a, tpr, sums, flip);" in text


def test_layer_norm_takes_turns():
    text = code("norm.cu")
    first = text.index("norm_fwd_rescaled(const NormArgs& a, int tpr, float* buf0, float* buf1, float* buf2)")
    body = text[first:text.index("norm_fwd_kernel", first)]
    used = re.findall(r"total\(([^()]*)\)", body)
    assert used == ["buf0", "buf1", "buf2", "f == LARGE ? buf1 : buf2"]
    for path in (["buf0", "buf1"], ["buf0", "buf1", "buf2", "buf1"], ["buf0", "buf1", "buf2"]):       # within range, LARGE, SMALL
        assert all(a != b for a, b in zip(path, path[1:] + ["buf0"]))                              # the next row's begin with buf0
    assert [b for b, _ in calls(text)] == ["buf", "sums[0]", "sums[1]", "sums[flip]"]
    # behind the loop, whose last sum is in sums[1]
    assert re.search(r"norm_fwd_rescaled<T, VEC, NV>\(a, tpr, sums\[0\], sums\[1\], sums\[2\]\)", text)
