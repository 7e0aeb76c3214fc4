"""api.layer_norm with each subset of its inputs that may want a gradient: every gradient against float64, and the same
bits whichever others are asked for with it.

Limits as in test_gpu_layer_norm.py: TERMS = d / 1024 + 72 roundings of 2^-24 a row, N / 152 + 90 for sums over rows, and
one rounding of the result (2^-8 for bfloat16)."""

import itertools

import numpy as np
import pytest
import torch

from memory_bounded_linear_gb300 import api
from oracle import token_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24


def _np(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [136, 515, 4096, 9000])
def test_subsets(cuda_lib, d, dt):
    N = 30
    g = torch.Generator().manual_seed(d)
    x, w, b, dy = (t.to(DT[dt]).cuda() for t in (torch.randn(N, d, generator=g), 1 + 0.2 * torch.randn(d, generator=g),
                                                torch.randn(d, generator=g), torch.randn(N, d, generator=g)))
    X, W, D = _np(x), _np(w), _np(dy)
    want = ref.layer_norm_backward(X, W, D)
    terms, rows = d / 1024 + 72, N / 152 + 90
    h, r = ref.layer_norm(X), 1 / np.sqrt(X.var(1, keepdims=True) + 1e-5)
    m = np.abs(D * W)
    limits = (4 * terms * U * r * (m + m.mean(1, keepdims=True) + np.abs(h) * (m * np.abs(h)).mean(1, keepdims=True)),
              (terms + rows) * U * (np.abs(D) * (1 + np.abs(h))).sum(0), rows * U * np.abs(D).sum(0))
    first = {}
    for wants in itertools.product([False, True], repeat=3):
        if not any(wants):
            continue
        leaves = [t.clone().requires_grad_(on) for t, on in zip((x, w, b), wants)]
        api.layer_norm(*leaves).backward(dy)
        for k, (t, on) in enumerate(zip(leaves, wants)):
            assert (t.grad is not None) == on
            if on:
                err = np.abs(_np(t.grad) - want[k])
                assert np.all(err <= limits[k] + (ROUND[dt] + 2 * U) * np.abs(want[k])), (wants, k)
                assert torch.equal(t.grad, first.setdefault(k, t.grad)), (wants, k)
    # a bias without a weight
    q = b.clone().requires_grad_(True)
    api.layer_norm(x, None, q).backward(dy)
    assert torch.equal(q.grad, first[2])


# widths on both sides of where rows no longer fit in registers, which differs by type, alignment and direction
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d", [4095, 4096, 4097, 8190, 8191, 8192, 8193, 8194, 8196, 16382, 16384, 16386, 16392])
def test_limits_of_the_registers(cuda_lib, d, dt):
    N = 3
    g = torch.Generator().manual_seed(d)
    x, w, b, dy = (t.to(DT[dt]).cuda() for t in (torch.randn(N, d, generator=g), 1 + 0.2 * torch.randn(d, generator=g),
                                                torch.randn(d, generator=g), torch.randn(N, d, generator=g)))
    X, W, B, D = _np(x), _np(w), _np(b), _np(dy)
    terms, rows = d / 1024 + 72, N / 152 + 90
    h = ref.layer_norm(X)
    want = ref.layer_norm(X, W, B)
    got = api.lce_layer_norm_forward(x, w, b)
    assert np.all(np.abs(_np(got) - want) <= terms * U * (1 + np.abs(h)) * np.abs(W) + (ROUND[dt] + 2 * U) * np.abs(want))
    r, m = 1 / np.sqrt(X.var(1, keepdims=True) + 1e-5), np.abs(D * W)
    limits = (4 * terms * U * r * (m + m.mean(1, keepdims=True) + np.abs(h) * (m * np.abs(h)).mean(1, keepdims=True)),
              (terms + rows) * U * (np.abs(D) * (1 + np.abs(h))).sum(0), rows * U * np.abs(D).sum(0))
    for t, v, limit in zip(api.lce_layer_norm_backward(x, w, b, dy)[:3], ref.layer_norm_backward(X, W, D), limits):
        assert np.all(np.abs(_np(t) - v) <= limit + (ROUND[dt] + 2 * U) * np.abs(v))
