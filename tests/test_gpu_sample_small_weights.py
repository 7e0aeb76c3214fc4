"""Sampling among weights of a few units of 2^-39 of the largest: which tokens are kept must not depend on where in the
row they lie, and must be what the definition says wherever integer weights can tell.

An integer weight is the exact one cut to an odd number, off by less than 2 units; tokens whose weight is 2 units and more
away from the floor are kept or dropped as in 64 bits.  With u = 0 the token drawn is the first one kept."""

import math

import numpy as np
import pytest
import torch

from memory_bounded_linear_gb300 import api
from oracle import token_ref as ref

pytestmark = pytest.mark.gpu
INF = float("inf")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _places(V):
    """(place of the small weight, of the largest): in the same 16 bytes, in a warp's neighbouring ones, chunks and CTAs apart."""
    return [(0, V - 1), (5, 6), (5, 37), (5, 300), (5, V // 2), (V // 3, V - 1), (V // 2, V // 2 + 1), (V - 2, V - 1), (1, 1000)]


def _rows(V, low, largest, dt):
    z = torch.full((len(_places(V)), V), -INF)
    for i, (a, b) in enumerate(_places(V)):
        z[i, a], z[i, b] = low, largest
    return z.to(DT[dt]).cuda(), torch.zeros(z.shape[0], device="cuda")


@pytest.mark.parametrize("dt,largest", [("f32", 0.0), ("bf16", 0.0), ("f32", 8192.0)])
@pytest.mark.parametrize("V", [2000, 20000, 151936])
def test_half_a_unit(cuda_lib, V, dt, largest):
    """2^-39.5 of the largest: the smallest weights there are belong to every sum, with a limit that keeps them or without."""
    for T in (1.0, 0.5):
        z, u = _rows(V, largest - 27.375 * T, largest, dt)         # exact in both types
        for s in (dict(), dict(top_k=600), dict(top_k=50), dict(min_p=1e-30), dict(top_k=600, min_p=1e-30)):
            tokens, _ = api.lce_sample(z, u, temperature=T, **s)
            for i, (a, b) in enumerate(_places(V)):
                assert ref.sample(z[i].double().cpu().numpy(), 0.0, T, s.get("top_k", 0), 1.0, s.get("min_p", 0.0))[0] == a
                assert tokens[i].item() == a, (T, s, i)


@pytest.mark.parametrize("min_p", [3e-12, 1e-11, 1e-10, 2.5e-10, 1e-9])
@pytest.mark.parametrize("V", [2000, 20000, 151936])
def test_floors_of_a_few_units(cuda_lib, V, min_p):
    floor = float(np.float32(min_p)) * 2.0 ** 39
    for units in (floor - 2.5, floor - 0.8, floor - 0.5, floor - 0.2, floor + 0.2, floor + 0.8, floor + 2.5):
        if units < 1:
            continue
        low = -math.log(2.0) * (39 - math.log2(units))
        for largest in (0.0, 8192.0):
            z, u = _rows(V, low + largest, largest, "f32")
            exact = 2.0 ** 39 * math.exp(float(z[0].double()[0]) - largest)
            for s in (dict(), dict(top_k=600), dict(top_k=50)):
                tokens, _ = api.lce_sample(z, u, min_p=min_p, **s)
                kept = [tokens[i].item() == a for i, (a, b) in enumerate(_places(V))]
                for i, (a, b) in enumerate(_places(V)):
                    assert tokens[i].item() in (a, b)
                assert len(set(kept)) == 1, (units, floor, s, kept)
                if abs(exact - floor) >= 2:
                    assert kept[0] == (exact > floor), (exact, floor, s)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_many_units_together(cuda_lib, dt):
    """150,000 tokens of half a unit each before the largest: they weigh 150,000 units of integer weights and 106,000 exactly, of
    2^39 both, below 2^-21 of the total; the draw is the largest for every u from there on, and one of them at 0."""
    V = 151936
    z = torch.full((1, V), -27.375).to(DT[dt]).cuda()
    z[0, V - 1] = 0.0
    u = torch.tensor([0.0, 2.0 ** -21, 0.5, 1 - 2.0 ** -24], device="cuda")
    for s in (dict(), dict(min_p=1e-30), dict(top_k=V - 1)):
        tokens, logprobs = api.lce_sample(z.expand(4, V).contiguous(), u, **s)
        # top-k leaves out the highest index of the equal ones
        assert tokens.tolist() == [0, V - 1, V - 1, V - 1], s
        assert logprobs[1:].abs().max() <= 2.0 ** -21
