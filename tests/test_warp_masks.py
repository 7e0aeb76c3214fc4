"""Warp-wide operations: every lane that a mask names has to reach the operation with that mask.  The kernels keep that
by full masks in loops and branches that all lanes of a warp take alike; a mask of the lanes that happen to run together
would promise nothing.  Read from the sources (CPU)."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "memory_bounded_linear_gb300", "csrc")
SOURCES = sorted(n for n in os.listdir(CSRC) if n.endswith((".cu", ".cuh", ".h")))


@pytest.mark.parametrize("path", SOURCES)
def test_masks_are_full(path):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, path)).read())
    assert "__activemask" not in text
    for m in re.finditer(r"__(?:ballot|any|all|shfl\w*|match\w*|reduce_\w+)_sync\(\s*([^,()]+)", text):
        assert m.group(1).strip() == "0xffffffffu", m.group(0)


def test_counts_of_digits_match_whole_warps():
    """The loop over a block's tokens has the same bound for all lanes of a warp."""
    text = open(os.path.join(CSRC, "lce_embed.cu")).read()
    body = text[text.index("embedding_count_kernel(const SortArgs a)"):text.index("embedding_sort_kernel(const SortArgs a)")]
    loop = re.search(r"for \(int64_t i = i0 \+ \(threadIdx\.x - lane\); i < i1; i \+= SORT_THREADS\) \{\n(.*?)\n  \}", body, re.S)
    assert loop is not None and "__match_any_sync(" in loop.group(1)
    assert "continue" not in loop.group(1) and "break" not in loop.group(1)
