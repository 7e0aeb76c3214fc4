"""An infinite total scales by 0, whatever the largest norm is; only a NaN total gives NaN everywhere."""

import pytest
import torch

from memory_bounded_linear_gb300 import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_norm", [0.0, 1.0, 3e38, float("inf")])
@pytest.mark.parametrize("norm", ["l2", "inf"])
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_infinite_total(cuda_lib, dt, norm, max_norm):
    g = [torch.ones(70_000, device="cuda"), torch.ones(9, device="cuda", dtype=dt)]
    g[1][3] = float("inf")
    total, out, _ = api.lce_clip_grad_norm(g, max_norm, norm=norm, out=[torch.empty_like(t) for t in g])
    assert total.item() == float("inf")
    assert not out[0].any()
    keep = [i for i in range(9) if i != 3]
    assert not out[1][keep].any() and torch.isnan(out[1][3])       # inf times 0


def test_no_limit(cuda_lib):
    """An infinite largest norm leaves finite gradients as they are."""
    g = [torch.randn(70_000, device="cuda"), torch.randn(9, device="cuda").bfloat16()]
    kept = [t.clone() for t in g]
    total, _, _ = api.lce_clip_grad_norm(g, float("inf"))
    assert torch.isfinite(total) and all(torch.equal(a, b) for a, b in zip(g, kept))


def test_square_sums_up_to_the_documented_size(cuda_lib):
    """Squares are summed in fp32 over a thread's share of a chunk: 2e18 in every place is still finite."""
    for dt in (torch.float32, torch.bfloat16):
        t = torch.full((200_003,), 2e18, device="cuda", dtype=dt)
        want = t[0].item() * 200_003 ** 0.5
        assert abs(api.lce_grad_norm([t])[0].item() - want) <= 2.0 ** -20 * want
