"""GELU of float32 far below zero, relative to its small value.

z reaches the activation exactly: one input feature times a weight of 1.  With s = sqrt(1/2):
* value z Phi(z) = z erfc(-z s) / 2.  The argument carries two roundings (s and the product), 1.3 2^-24
  together, which erfc turns into z^2 + 2 times as much; erfcf is good to 4 units in the last place
  (8 2^-24), the product is rounded once: (1.3 (z^2 + 2) + 9) 2^-24, below (z^2 + 10) 2^-23.
* derivative Phi(z) + z exp(-z^2/2) / sqrt(2 pi): the first term is at most 0.11 of the second for
  z <= -3, so the sum loses little; the exponent z^2/2 carries one rounding, expf two units, the products
  three roundings, Phi as above: below (z^2 + 16) 2^-23."""

import math

import pytest
import torch

from memory_bounded_linear_gb300 import api

pytestmark = pytest.mark.gpu


def _inputs(N):
    z = torch.linspace(-8.0, -3.0, N, dtype=torch.float64).float()
    x, w = torch.zeros(N, 8), torch.zeros(8, 8)
    x[:, 0], w[0, 0] = z, 1.0
    return z.double(), x.cuda(), w.cuda()


def _phi(z):
    return torch.tensor([0.5 * math.erfc(-v * math.sqrt(0.5)) for v in z.tolist()], dtype=torch.float64)


@pytest.mark.parametrize("N", [40, 4500])        # dot products, tiles
def test_value(cuda_lib, N):
    z, x, w = _inputs(N)
    want = z * _phi(z)
    y = api.lce_linear_forward(x, w, activation="gelu")[0][:, 0].cpu().double()
    err = ((y - want) / want).abs()
    assert torch.all(err <= (z * z + 10) * 2.0 ** -23), err.max()
    one = torch.zeros(8, 8)
    one[0, 0] = 1.0
    h = api.lce_gated_forward(torch.cat([x, torch.ones_like(x)], 1), torch.cat([w, torch.zeros_like(w)], 1),
                              torch.cat([torch.zeros_like(w), one.cuda()], 1), activation="gelu")[0][:, 0]
    err = ((h.cpu().double() - want) / want).abs()
    assert torch.all(err <= (z * z + 10) * 2.0 ** -23), err.max()


@pytest.mark.parametrize("N", [40, 4500])
def test_derivative(cuda_lib, N):
    z, x, w = _inputs(N)
    want = _phi(z) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    dy = torch.zeros(N, 8, device="cuda")
    dy[:, 0] = 1.0
    dx = api.lce_linear_backward(x, w, None, dy, activation="gelu", parts="dx")[0][:, 0].cpu().double()
    err = ((dx - want) / want).abs()
    assert torch.all(err <= (z * z + 16) * 2.0 ** -23), err.max()
