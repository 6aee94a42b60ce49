"""Waits that have to end alike for every thread, read from the kernels' sources.

What goes wrong without them is a hang or a race on memory, which no test may cause on a GPU;
so these look at the code itself."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "verifiable_quantize_rows_gb300", "csrc")


def source(name):
    """The file without its comments."""
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def body(text, head):
    """What stands between the braces that follow `head`."""
    at = text.index("{", text.index(head))
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == "{") - (text[i] == "}")
        if not depth:
            return text[at + 1:i]
    raise AssertionError(head)


def test_the_sums_warps_leave_together():
    """The warps that take sums meet at a barrier of their own in every round.  Another role may
    set the abort flag at any time, so a thread that read it for itself could leave while its
    neighbours go on to that barrier for good: one warp waits, and all go by what the barrier
    itself answers."""
    kernel = body(source("wcols.cu"), "wcols_few_kernel(const")
    sums = kernel[kernel.index("} else {", kernel.index("const int row0 = lane / 16")):]   # the last role
    assert "bar.sync 1" in sums and "atomicAdd" in sums
    assert "abort_flag" not in sums
    assert "if (warp == 0) came = all_wait(&sum_full[c & 1], c >> 1 & 1);" in sums
    assert "if (!(ok = sums_barrier_all(came))) break;" in sums     # the barrier's own answer, one for all
    assert sums.count("all_wait") == 1 and "barrier.cta.red.and.pred" in body(source("wcols.cu"), "bool sums_barrier_all(bool x)")


def test_no_block_of_a_grid_launched_beside_another_ends_before_it():
    """A grid launched while the one before it still runs has to wait for it in every block: were
    all to leave early (a join where no token is there), the next call could begin to write the
    workspace while the first grid is still at it."""
    for name, head in (("kv8_more.cu", "kv8_join_lists_kernel(const"), ("kv8.cu", "kv8_join_kernel(const")):
        kernel = body(source(name), head)
        assert "return;" not in kernel[:kernel.index("griddep_wait();")], name
    kernel = body(source("quantize.cu"), "i8_cols_to_half_kernel(const")
    assert "return" not in re.sub(r"return \*reinterpret_cast[^;]*;", "", kernel) and kernel.rstrip().endswith("griddep_wait();")
    # the tiles' kernel: a block without rows leaves at once, which those of a prefix are not; one without tiles waits
    kernel = body(source("kv8_tiles.cuh"), "kv8_tiles_kernel(const")
    early = body(kernel, "if (tiles == 0 && split > 0)")
    assert early.index("if (PREFIX) griddep_wait();") < early.index("return;")
