"""The fp32 limit against mistakes planted in a float64 model of the six part products (CPU)."""

import itertools

import numpy as np
import pytest
import torch

from .ffn_limits import F32

SIX = [(2, 0), (0, 2), (1, 1), (1, 0), (0, 1), (0, 0)]


def _parts(x):
    out, rest = [], x
    for _ in range(3):
        p = rest.to(torch.bfloat16).float()
        out.append(p.double().numpy())
        rest = rest - p
    assert not rest.any()                         # 8 + 8 + 8 bits hold a float32 value
    return out


@pytest.mark.parametrize("K", [256, 1024, 4096])
def test_a_missing_part_product_is_seen(K):
    g = torch.Generator().manual_seed(K)
    x, w = torch.randn(48, K, generator=g), torch.randn(40, K, generator=g) * K ** -0.5
    want = x.double().numpy() @ w.double().numpy().T
    a, b = _parts(x), _parts(w)

    def error(pairs):
        got = sum(a[i] @ b[j].T for i, j in pairs)
        return np.linalg.norm(got - want) / np.linalg.norm(want)
    assert error(SIX) < 0.1 * F32
    for lost in range(1, 4):
        for gone in itertools.combinations(SIX, lost):
            assert error([p for p in SIX if p not in gone]) > 1.5 * F32, gone
