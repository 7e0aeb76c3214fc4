"""Grids of normalisation go by the number of SMs that the device reports: the one number of SMs that is written out bounds
the workspace, whose size is asked for without a device.  Read from the source (CPU)."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "memory_bounded_linear_gb300", "csrc")


def test_no_grid_has_a_number_of_sms_written_out():
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "lce_norm.cu")).read())
    bound = text[text.index("int64_t max_parts("):text.index("struct NormArgs")]
    assert "152" in bound and "152" not in text.replace(bound, "")
    assert len(re.findall(r"\b(?:forward|backward)_rows<[^;]*num_sms", text)) >= 20
