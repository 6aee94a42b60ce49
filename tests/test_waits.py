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
    neighbours go on to that barrier for good: only one thread may read it, and all go by what
    that one wrote before the barrier."""
    kernel = body(source("wcols.cu"), "wcols_few_kernel(const")
    sums = kernel[kernel.index("} else {", kernel.index("const int row0 = lane / 16")):]   # the last role
    assert "bar.sync 1" in sums and "atomicAdd" in sums
    one = body(sums, "if (warp == 0)")
    assert "abort_flag" in one and "lane == 0" in one
    assert sums.count("abort_flag") == one.count("abort_flag")
    loop = sums[sums.index(one) + len(one):]
    assert loop.index("bar.sync 1") < loop.index("break;")        # decided behind the barrier, by its word
