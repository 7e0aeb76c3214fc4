"""The timeout path of the feed-forward kernels, without faulting or hanging the GPU: a launch whose
operands are withheld gives up after its 2 s wait limit, reports LCE_ERR_TIMEOUT through the
workspace, and leaves the context usable."""

import time

import pytest
import torch

from memory_bounded_linear_gb300 import api
from memory_bounded_linear_gb300._lib import LceError

pytestmark = pytest.mark.gpu

# N, d, F: few tokens in clusters of 8 and alone; tiles cut over clusters, one wave, tiles by tickets
CASES = [(4, 1024, 256), (4, 64, 256), (300, 1024, 256), (600, 128, 4096), (20000, 64, 5120)]


def _inputs(N, d, F):
    g = torch.Generator(device="cuda").manual_seed(N)
    return [(torch.randn(*s, generator=g, device="cuda") * k).bfloat16()
            for s, k in (((N, d), 1.0), ((F, d), d ** -0.5), ((F, d), d ** -0.5), ((N, F), 1.0))]


def _times_out(lib, call):
    torch.cuda.synchronize()
    try:
        assert lib.lce_test_inject_stall(1) == 0
        t0 = time.monotonic()
        ws = call()[-1]
        with pytest.raises(LceError) as e:
            api.lce_check_error(ws)
        assert e.value.name == "LCE_ERR_TIMEOUT"
        assert 1.5 < time.monotonic() - t0 < 60.0
    finally:
        lib.lce_test_inject_stall(0)


@pytest.mark.parametrize("N,d,F", CASES)
def test_forward(cuda_lib, N, d, F):
    x, wg, wu, _ = _inputs(N, d, F)
    want, ws = api.lce_gated_forward(x, wg, wu)
    api.lce_check_error(ws)
    _times_out(cuda_lib, lambda: api.lce_gated_forward(x, wg, wu, workspace=ws))
    got, ws = api.lce_gated_forward(x, wg, wu, workspace=ws)     # the same workspace works again
    api.lce_check_error(ws)
    assert torch.equal(got, want)


@pytest.mark.parametrize("N,d,F", CASES[2:])
def test_backward(cuda_lib, N, d, F):
    x, wg, wu, dh = _inputs(N, d, F)
    want = api.lce_gated_backward(x, wg, wu, dh)
    api.lce_check_error(want[-1])
    _times_out(cuda_lib, lambda: api.lce_gated_backward(x, wg, wu, dh, workspace=want[-1]))
    got = api.lce_gated_backward(x, wg, wu, dh, workspace=want[-1])
    api.lce_check_error(got[-1])
    assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
