"""The example that runs the operators together: one training step's loss and gradients against a
float64 computation of the same model, falling losses, and decoding token by token."""

import os
import sys

import numpy as np
import pytest
import torch

import oracle
from oracle import ffn_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import block_and_head as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def _np(t):
    return t.detach().cpu().double().numpy()


# bf16: h, y and the gradients between the operators are rounded to bf16 (2^-9 each); a gradient of
# the block passes five such roundings: 5 * 2^-9, taken as 2^-6.  fp32: 2e-5 per operator, 1e-4.
@pytest.mark.parametrize("dt,tol", [("bf16", 2.0 ** -6), ("f32", 1e-4)])
def test_one_step(cuda_lib, dt, tol):
    dtype = {"bf16": torch.bfloat16, "f32": torch.float32}[dt]
    torch.manual_seed(3)
    m = ex.BlockAndHead(72, 200, 520, device="cuda", dtype=dtype)
    x = torch.randn(333, 72, device="cuda").to(dtype)
    labels = torch.randint(0, 520, (333,), device="cuda")
    loss = m.loss(x, labels)
    loss.backward()
    X, G, U, D, B, W = (_np(t) for t in (x, m.block.gate, m.block.up, m.block.down, m.block.bias, m.head))
    h = ref.gated(X, G, U)
    y = ref.linear(h, D, B, X)
    r = oracle.forward_backward(y, W, labels.cpu().numpy())
    assert abs(loss.item() - r["loss"]) <= tol * abs(r["loss"])
    dh, dd, db = ref.linear_backward(h, D, B, r["dH"])
    _, dg, du = ref.gated_backward(X, G, U, dh)
    for p, want in ((m.head, r["dW"]), (m.block.down, dd), (m.block.bias, db), (m.block.gate, dg),
                    (m.block.up, du)):
        err = np.linalg.norm(_np(p.grad) - want) / np.linalg.norm(want)
        assert err <= tol, err


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_example_runs(cuda_lib, dt):
    losses, norms, together, one_by_one = ex.main(["--tokens", "400", "--width", "256", "--ffn", "520",
                                                   "--vocab", "1000", "--steps", "12", "--dtype", dt])
    assert all(np.isfinite(losses)) and all(np.isfinite(norms))
    assert losses[-1] < 0.9 * losses[0]
    assert torch.equal(together, one_by_one)
