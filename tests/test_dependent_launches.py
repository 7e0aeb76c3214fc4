"""Kernels launched while the previous one drains: what makes that safe is that every one of them waits for
it before it touches memory of the caller.  Read from the sources (CPU)."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "memory_bounded_linear_gb300", "csrc")
FILES = ["lce_gradnorm.cu", "lce_ffn_few.cu", "lce_ffn_simt.cu", "lce_ffn_tc.cu"]


def _kernels(path):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, path)).read())
    for m in re.finditer(r"__global__\s+void\b", text):
        begin = text.index("{", text.index(") {", m.end()))
        depth, i = 1, begin + 1
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield re.search(r"(\w+_kernel)\(", text[m.end():begin]).group(1), text[begin:i]


# accesses of memory that another launch may write: loads and stores through a kernel's pointers, the
# helpers that make them, TMA, atomics
TOUCHES = re.compile(r"\bload<|\bvisit<|\bscale<|\btotal_of<|\bpart\[|\*\s*total\b|__ldg\(|__ldcs\(|\*p\.err\b|\*err\b|\*flags\b"
                     r"|\btma_(load|store)|\batomic\w+\(|\bp\.header\[|\bcopy16_async\(|\bfinish<|\bp\.bias\[|\bout\[")


def test_every_kernel_is_found():
    names = [k for f in FILES for k, _ in _kernels(f)]
    assert sorted(names) == sorted(["norm_kernel", "total_kernel", "scale_kernel", "ffn_few_kernel", "few_f32_kernel",
                                    "column_sum_kernel", "pack_kernel", "ffn_tc_kernel"])


@pytest.mark.parametrize("path", FILES)
def test_waits_before_it_touches_memory(path):
    for name, body in _kernels(path):
        assert body.count("wait_for_previous()") == 1, name
        waits = body.index("wait_for_previous()")
        early = TOUCHES.search(body[:waits])
        assert early is None, (name, early.group(0))
        assert "launch_dependents()" not in body[:waits], name
