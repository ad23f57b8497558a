"""What can be read off the dense block's kernels without a GPU."""
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "sparse_moe_ffn_route_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def braces(text, start):
    """The block that opens at or after `start`."""
    first = text.index("{", start)
    depth = 0
    for i in range(first, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[first:i + 1]
    raise AssertionError("unbalanced")


def test_epilogue_warps_leave_their_waits_together():
    """Whole warps run the epilogue, with warp-wide tensor-memory loads, votes and shuffles: a
    wait there, and the abort flag, must give every lane the same answer."""
    text = source("glu_gemm.cu")
    loop = braces(text, text.index("for (", text.index("const int par = (warp - 2) >> 2;")))
    head = text[text.index("for (", text.index("const int par = (warp - 2) >> 2;")):text.index(loop)]
    assert "tcgen05" not in head and "tmem_ld" in loop
    assert "tc::mbar_wait(" not in loop and loop.count("warp_wait(") >= 2
    for text_part in (head, loop):
        for m in re.finditer(r"\*abort", text_part):
            assert "__all_sync(" in text_part[:m.start()][-40:], text_part[max(0, m.start() - 60):m.end()]
    helper = braces(text, text.index("bool warp_wait("))
    assert "__all_sync(0xffffffffu, tc::mbar_wait(" in helper
