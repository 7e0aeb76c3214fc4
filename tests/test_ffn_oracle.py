"""The float64 definitions of the feed-forward operators, pinned by differences and closed forms."""

import math

import numpy as np
import pytest

from oracle import ffn_ref as ref

STEP = 1e-5
# Central differences in float64: truncation STEP^2 |f'''| / 6 (a few 1e-11 here) and rounding
# 1e-16 |f| / STEP (about 1e-10 for |f| up to 10): 1e-8 leaves two orders of magnitude.
TOL = 1e-8


def _difference(f, x):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        hi, lo = x.copy(), x.copy()
        hi[i] += STEP
        lo[i] -= STEP
        g[i] = (f(hi) - f(lo)) / (2 * STEP)
    return g


@pytest.mark.parametrize("a", ref.ACTIVATIONS)
def test_activation_gradient_matches_differences(a):
    z = np.linspace(-6.05, 6.05, 122)  # no point within a step of 0, where relu has a corner
    d = (ref.act(z + STEP, a) - ref.act(z - STEP, a)) / (2 * STEP)
    assert np.max(np.abs(d - ref.act_grad(z, a))) <= TOL


@pytest.mark.parametrize("a", ref.ACTIVATIONS)
def test_gradients_match_differences(a):
    r = np.random.RandomState(1)
    x, wg, wu = r.randn(3, 4), r.randn(5, 4), r.randn(5, 4)
    b, dy = r.randn(5), r.randn(3, 5)
    dx, dwg, dwu = ref.gated_backward(x, wg, wu, dy, a)
    assert np.max(np.abs(dx - _difference(lambda t: np.sum(ref.gated(t, wg, wu, a) * dy), x))) <= TOL
    assert np.max(np.abs(dwg - _difference(lambda t: np.sum(ref.gated(x, t, wu, a) * dy), wg))) <= TOL
    assert np.max(np.abs(dwu - _difference(lambda t: np.sum(ref.gated(x, wg, t, a) * dy), wu))) <= TOL
    dx, dw, db = ref.linear_backward(x, wg, b, dy, a)
    f = lambda xx, ww, bb: np.sum(ref.linear(xx, ww, bb, None, a) * dy)  # noqa: E731
    assert np.max(np.abs(dx - _difference(lambda t: f(t, wg, b), x))) <= TOL
    assert np.max(np.abs(dw - _difference(lambda t: f(x, t, b), wg))) <= TOL
    assert np.max(np.abs(db - _difference(lambda t: f(x, wg, t), b))) <= TOL


def test_closed_forms():
    assert ref.act(np.array([0.0]), "silu")[0] == 0.0
    assert ref.act(np.array([1.0]), "gelu")[0] == pytest.approx(0.8413447460685429, rel=1e-12)
    assert ref.act(np.array([2.0]), "silu")[0] == pytest.approx(2 / (1 + math.exp(-2)), rel=1e-14)
    total, out = ref.clip([np.array([3.0]), np.array([4.0])], 1.0)
    assert total == 5.0 and out[0][0] == pytest.approx(0.6, rel=1e-6)
    total, out = ref.clip([np.array([0.3]), np.array([-0.4])], 1.0)
    assert total == pytest.approx(0.5) and out[1][0] == -0.4
    assert ref.grad_norm([np.array([1.0, -7.0]), np.array([])], "inf") == 7.0
