"""What an entry point writes into a caller's tensor, autograd knows of: a tensor that was saved for a
backward pass and then overwritten is an error there, not a wrong gradient."""

import pytest
import torch

from memory_bounded_linear_gb300 import api

pytestmark = pytest.mark.gpu


def _saved(*shape):
    t = torch.randn(*shape, device="cuda", requires_grad=True)
    e = t.exp()                                  # exp saves its result
    return e, e.detach()                         # the same memory, outside the graph


def _refuses(e):
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        e.sum().backward()


@pytest.mark.parametrize("N", [4, 300])
def test_out_of_products(cuda_lib, N):
    x, w = torch.randn(N, 64, device="cuda"), torch.randn(96, 64, device="cuda")
    for call in (lambda o: api.lce_linear_forward(x, w, out=o), lambda o: api.lce_gated_forward(x, w, w, out=o),
                 lambda o: api.lce_linear_forward(x, w, None, o, out=o)):
        e, o = _saved(N, 96)
        before = o._version
        call(o)
        assert o._version == before + 1
        _refuses(e)


def test_clipped_gradients(cuda_lib):
    e, g = _saved(1000)
    api.lce_clip_grad_norm([g], 1.0)
    _refuses(e)
    e, o = _saved(1000)
    g = torch.randn(1000, device="cuda")
    before = g._version
    api.lce_clip_grad_norm([g], 1.0, out=[o])
    assert g._version == before                  # read only
    _refuses(e)
    e, g = _saved(1000)
    api.lce_grad_norm([g])
    e.sum().backward()                           # read only


def test_tensors_without_versions(cuda_lib):
    with torch.inference_mode():
        x, w = torch.randn(4, 64, device="cuda"), torch.randn(96, 64, device="cuda")
        out = torch.empty(4, 96, device="cuda")
        assert api.lce_linear_forward(x, w, out=out)[0] is out
        api.lce_clip_grad_norm([x], 1.0)
    assert torch.isfinite(out).all()
