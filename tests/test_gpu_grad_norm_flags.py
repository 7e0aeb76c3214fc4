"""The error flags of a clipping call's workspace: the call clears them, whatever was in the memory, so
that lce_check_error reports on this call."""

import pytest
import torch

from memory_bounded_linear_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes", [[5], [300_001, 7, 0, 12], [3] * 700, [0, 0]])
@pytest.mark.parametrize("norm", ["l2", "inf"])
def test_flags_are_cleared(cuda_lib, sizes, norm):
    grads = [torch.ones(n, device="cuda") for n in sizes]
    for call in (lambda ws: api.lce_grad_norm(grads, norm=norm, workspace=ws),
                 lambda ws: api.lce_clip_grad_norm(grads, 1.0, norm=norm, workspace=ws)):
        ws = torch.full((1 << 16,), 0xff, dtype=torch.uint8, device="cuda")
        api.lce_check_error(call(ws)[-1])


def test_flags_of_an_earlier_call(cuda_lib):
    """A workspace that the head flagged a bad label in."""
    H, W = torch.zeros(8, 64, device="cuda"), torch.zeros(300, 64, device="cuda")
    y = torch.full((8,), 300, dtype=torch.int64, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    api.lce_forward(H, W, y, strip_V=256, workspace=ws)
    with pytest.raises(RuntimeError, match="LABEL"):
        api.lce_check_error(ws)
    api.lce_clip_grad_norm([torch.ones(9, device="cuda")], 1.0, workspace=ws)
    api.lce_check_error(ws)
