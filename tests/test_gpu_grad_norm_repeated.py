"""The same memory twice in a list of gradients.  Scaling it from two places at once would leave some
values scaled once and some twice, so the list call refuses it; over parameters it counts once."""

import pytest
import torch

from memory_bounded_linear_gb300 import api

pytestmark = pytest.mark.gpu


def test_parameters_that_appear_twice(cuda_lib):
    p = [torch.nn.Parameter(torch.randn(300, 700, device="cuda")), torch.nn.Parameter(torch.randn(11, device="cuda"))]
    for t in p:
        t.grad = torch.randn_like(t)
    kept = [t.grad.clone() for t in p]
    want = torch.cat([k.flatten() for k in kept]).double().norm()
    total = api.clip_grad_norm_([p[0], p[1], p[0]], 1.0)
    assert abs(total.item() - want.item()) <= 2.0 ** -20 * want.item()
    for t, k in zip(p, kept):
        assert torch.allclose(t.grad, k / want.float(), rtol=1e-5, atol=0)
    tied = [torch.nn.Parameter(torch.zeros(5, device="cuda")) for _ in range(2)]
    tied[0].grad = torch.full((5,), 2.0, device="cuda")
    tied[1].grad = tied[0].grad                                     # one gradient in two parameters
    assert abs(api.clip_grad_norm_(tied, 1.0).item() - 20 ** 0.5) <= 1e-5
    assert torch.allclose(tied[0].grad, torch.full((5,), 2 / 20 ** 0.5, device="cuda"), rtol=1e-5)


def test_overlapping_outputs_are_refused(cuda_lib):
    a, b = torch.randn(1000, device="cuda"), torch.randn(1000, device="cuda")
    kept = a.clone()
    o = torch.empty(2000, device="cuda")
    for grads, out in (([a, b, a], None),                          # in place, twice
                       ([a, a[10:20]], None),                       # a part of it
                       ([a[:600], a[599:]], None),
                       ([a, b], [o[:1000], o[999:1999]]),           # one value shared
                       ([a, b], [o[:1000], a]),                     # another's input
                       ([a, b], [b, a]),
                       ([a[:500]], [a[1:501]]),                     # its own input, shifted
                       ([a, a], [a, o[:1000]])):
        with pytest.raises(ValueError, match="overlap"):
            api.lce_clip_grad_norm(grads, 1.0, out=out)
    assert torch.equal(a, kept)
    # neighbours, own inputs, empty arrays and inputs that repeat beside outputs of their own are fine
    api.lce_clip_grad_norm([a[:600], a[600:], a[600:600], b], 1e9)
    api.lce_clip_grad_norm([a, b], 1e9, out=[a, o[:1000]])
    total, _, _ = api.lce_clip_grad_norm([a, a], 1e9, out=[o[:1000], o[1000:]])
    assert torch.equal(o[:1000], kept) and torch.equal(o[1000:], kept)
    assert abs(total.item() - 2 ** 0.5 * kept.double().norm().item()) <= 2.0 ** -19 * total.item()
    assert api.lce_grad_norm([a, a])[0].item() == total.item()
