"""Every kernel of the feed-forward operators at limits (ffn_limits.py) that show a missing part product,
a lost piece of a sum or a chunk that was not written: norms, and element by element over the whole
result.  Against plain products in float64 on the GPU."""

import pytest
import torch

from memory_bounded_linear_gb300 import api

from .ffn_limits import BF16, BF16_TERMS, F32, F32_TWO

pytestmark = pytest.mark.gpu


def _check(got, want, limit, spread, what):
    """limit: of the norm; spread: of each element and the rms."""
    want = want.detach()
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    err = (got.double() - want).abs()
    rel = (err.norm() / want.norm()).item()
    rms = want.norm() / want.numel() ** 0.5
    worst = (err / (want.abs() + rms)).max().item()
    assert rel <= limit, (what, rel)
    assert worst <= spread, (what, worst)


def _check_gradient(got, want, squares, what):
    """bf16; squares: the sum of the squared terms of each element."""
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    err = (got.double() - want).abs()
    limit = BF16 * want.abs() + BF16_TERMS * squares.sqrt()
    assert (err <= limit).all(), (what, (err / limit.clamp_min(1e-300)).max().item())


def _rand(N, d, F, dtype):
    g = torch.Generator(device="cuda").manual_seed(N + 3 * d + 7 * F)
    return [(torch.randn(*s, generator=g, device="cuda") * k).to(dtype)
            for s, k in (((N, d), 1.0), ((F, d), d ** -0.5), ((F, d), d ** -0.5), ((F,), 1.0), ((N, F), 1.0))]


# dot products of one to eight warps a sum; tiles of both widths, alone and in clusters of two and four
# pairs, several waves, taken as tickets, sums of one step and of many, ragged everywhere
F32_SHAPES = [(1, 2048, 516), (3, 4100, 260), (8, 2048, 2052), (21, 516, 1028), (48, 2052, 260), (333, 1028, 1004),
              (49, 2052, 2052), (130, 260, 4100), (601, 260, 1004), (500, 4096, 516), (2000, 1000, 2000),
              (1000, 2048, 8192), (4100, 68, 132), (8192, 132, 260)]


@pytest.mark.parametrize("N,d,F", F32_SHAPES)
def test_f32(cuda_lib, N, d, F):
    x, w, wu, b, dy = _rand(N, d, F, torch.float32)
    X, W, U, B, D = (t.double() for t in (x, w, wu, b, dy))
    z, u = X @ W.t(), X @ U.t()
    y, ws = api.lce_linear_forward(x, w)
    api.lce_check_error(ws)
    _check(y, z, F32, 8 * F32, "y")
    _check(api.lce_linear_forward(x, w, b, dy)[0], z + B + D, F32, 8 * F32, "y + bias + residual")
    _check(api.lce_gated_forward(x, w, wu, activation="none")[0], z * u, F32_TWO, 8 * F32_TWO, "h")
    dx, dw, db, _ = api.lce_linear_backward(x, w, b, dy)
    _check(dx, D @ W, F32, 8 * F32, "dx")
    _check(dw, D.t() @ X, F32, 8 * F32, "dw")
    _check(db, D.sum(0), F32, 8 * F32, "db")
    dx, dwg, dwu, ws = api.lce_gated_backward(x, w, wu, dy, activation="none")
    api.lce_check_error(ws)
    dg, du = D * u, D * z
    _check(dx, dg @ W + du @ U, F32_TWO, 8 * F32_TWO, "gated dx")
    _check(dwg, dg.t() @ X, F32_TWO, 8 * F32_TWO, "dwg")
    _check(dwu, du.t() @ X, F32_TWO, 8 * F32_TWO, "dwu")


BF16_SHAPES = [(1, 2048, 1032), (4, 16384, 520), (40, 1024, 11008), (150, 8192, 2048), (300, 200, 264),
               (600, 9216, 520), (777, 1032, 1096), (2600, 1032, 2600), (4096, 1024, 4096), (16384, 128, 264),
               (20000, 64, 5128)]


@pytest.mark.parametrize("N,d,F", BF16_SHAPES)
def test_bf16(cuda_lib, N, d, F):
    x, w, wu, b, dy = _rand(N, d, F, torch.bfloat16)
    X, W, U, B, D = (t.double() for t in (x, w, wu, b, dy))
    z, u = X @ W.t(), X @ U.t()
    s = torch.sigmoid(z)
    h, ws = api.lce_gated_forward(x, w, wu)
    api.lce_check_error(ws)
    _check(h, z * s * u, BF16, BF16, "h")
    dg, du = D * u * (s + z * s * (1 - s)), D * z * s
    del z, u, s
    dx, dwg, dwu, ws = api.lce_gated_backward(x, w, wu, dy)
    api.lce_check_error(ws)
    _check_gradient(dx, dg @ W + du @ U, dg ** 2 @ W ** 2 + du ** 2 @ U ** 2, "gated dx")
    _check_gradient(dwg, dg.t() @ X, (dg ** 2).t() @ X ** 2, "dwg")
    _check_gradient(dwu, du.t() @ X, (du ** 2).t() @ X ** 2, "dwu")
    del dg, du, dx, dwg, dwu
    z = X @ W.t() + B
    s = torch.sigmoid(z)
    _check(api.lce_linear_forward(x, w, b, dy, activation="silu")[0], z * s + D, BF16, BF16, "y")
    dz = D * (s + z * s * (1 - s))
    dx, dw, db, _ = api.lce_linear_backward(x, w, b, dy, activation="silu")
    _check_gradient(dx, dz @ W, dz ** 2 @ W ** 2, "dx")
    _check_gradient(dw, dz.t() @ X, (dz ** 2).t() @ X ** 2, "dw")
    _check_gradient(db, dz.sum(0), (dz ** 2).sum(0), "db")
