"""Layer normalisation of rows whose squared differences leave fp32: finite values, a sum that is not.  Such a row is NaN
whichever kernel its width, type and alignment lead to, never the bias alone; its neighbours are right.

The limits of what is right are those of test_gpu_layer_norm.py: TERMS = d / 1024 + 72 roundings of 2^-24 of 1 + |x^|,
times |w|, and one rounding of the result (2^-8 for bfloat16)."""

import numpy as np
import pytest
import torch

from memory_bounded_linear_gb300 import api
from oracle import token_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ROUND = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24

# width, elements before the row: rows held in registers by 16 bytes, 4 bytes and single elements, and rows read again
PLACES = [(264, 0), (1003, 1), (4096, 0), (4100, 1), (9000, 0), (9000, 1), (9000, 2), (16384, 0), (20000, 0), (20001, 1)]


def _np(t):
    return t.detach().cpu().double().numpy()


def _rows(N, d, off, dt, seed=0):
    g = torch.Generator().manual_seed(seed + d + off)
    buf = torch.zeros(N, d + 16, dtype=DT[dt], device="cuda")
    x = buf[:, off:off + d]
    x.copy_(torch.randn(N, d, generator=g))
    w, b = ((1 + 0.2 * torch.randn(d, generator=g)).to(DT[dt]).cuda() for _ in range(2))
    return x, w, b, torch.randn(N, d, generator=g).to(DT[dt]).cuda()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d,off", PLACES)
def test_overflow_is_nan(cuda_lib, d, off, dt):
    x, w, b, dy = _rows(5, d, off, dt)
    sign = torch.where(torch.arange(d, device="cuda") % 2 == 0, 1.0, -1.0)
    x[1] = (1e20 * sign).to(DT[dt])                                # mean 0, or nearly
    x[3, d // 2] = 3e19                                            # one value far off
    y = api.lce_layer_norm_forward(x, w, b)
    assert torch.isnan(y[[1, 3]]).all()
    dx, dw, db, ws = api.lce_layer_norm_backward(x, w, b, dy)
    api.lce_check_error(ws)
    assert torch.isnan(dx[[1, 3]]).all() and torch.isnan(dw).all() and torch.isfinite(db).all()
    fine = [0, 2, 4]
    want = ref.layer_norm(_np(x[fine]), _np(w), _np(b))
    limit = (d / 1024 + 72) * U * (1 + np.abs(ref.layer_norm(_np(x[fine])))) * np.abs(_np(w)) + \
        (ROUND[dt] + 2 * U) * np.abs(want)
    assert np.all(np.abs(_np(y[fine]) - want) <= limit) and torch.isfinite(dx[fine]).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("d,off", PLACES)
def test_large_values_that_fit(cuda_lib, d, off, dt):
    """Differences of up to 5e15: their squares add up to 2.5e31 d at most, 5e35 here."""
    x, w, b, dy = _rows(4, d, off, dt, seed=1)
    x.mul_(1e15)
    x[0].clamp_(-5e15, 5e15)
    y = api.lce_layer_norm_forward(x, w, b)
    want = ref.layer_norm(_np(x), _np(w), _np(b))
    limit = (d / 1024 + 72) * U * (1 + np.abs(ref.layer_norm(_np(x)))) * np.abs(_np(w)) + (ROUND[dt] + 2 * U) * np.abs(want)
    assert np.all(np.abs(_np(y) - want) <= limit)
    dx, dw, db, _ = api.lce_layer_norm_backward(x, w, b, dy)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all() and torch.isfinite(db).all()
