"""Lists of gradients and outputs from any iterable."""

import pytest
import torch

from memory_bounded_linear_gb300 import api

pytestmark = pytest.mark.gpu


def test_outputs_from_an_iterator(cuda_lib):
    """Gradients and outputs may come from any iterable; the outputs come back."""
    a, b = torch.randn(1000, device="cuda"), torch.randn(7, device="cuda")
    outs = [torch.empty_like(a), torch.empty_like(b)]
    _, got, _ = api.lce_clip_grad_norm((t for t in (a, b)), 1e9, out=(t for t in outs))
    assert len(got) == 2 and got[0] is outs[0] and got[1] is outs[1] and torch.equal(outs[0], a)
