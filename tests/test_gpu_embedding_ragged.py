"""The embedding's gradient where the last warp of the last block of the digit counts is not full: more than 8,192 positions,
N modulo 1,024 and modulo 32 from one to all but one.

Limits as in test_gpu_embedding.py: a token's n terms one after the other take n + 10 roundings of 2^-24 of the sum of
their magnitudes at most, the scale and the result one each (2^-8 for bfloat16)."""

import numpy as np
import pytest
import torch

from memory_bounded_linear_gb300 import api
from oracle import token_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("how", ["zipf", "one", "padded", "bad"])
@pytest.mark.parametrize("N", [8193, 8223, 8224, 8225, 9215, 9216, 9217, 10239, 66561, 66591])
def test_ragged_positions(cuda_lib, N, how):
    V, d = 1500, 8
    rng = np.random.RandomState(N)
    t = np.minimum(rng.zipf(1.2, N) - 1, V - 1)
    if how == "one":
        t[:] = V - 1
    elif how == "padded":
        t[rng.rand(N) < 0.6] = -100
        t[-5:] = -100
    elif how == "bad":
        t[rng.rand(N) < 0.1] = V
        t[-1] = -7
    tokens = torch.from_numpy(t.astype(np.int64)).cuda()
    g = torch.Generator().manual_seed(N)
    dy = torch.randn(N, d, generator=g).cuda()
    got, ws = api.lce_embedding_backward(tokens, dy, V, scale=0.5)
    if how == "bad":
        with pytest.raises(Exception, match="LABEL"):
            api.lce_check_error(ws)
    else:
        api.lce_check_error(ws)
    D = dy.cpu().double().numpy()
    want = ref.embedding_backward(t, D, V, 0.5)
    size = ref.embedding_backward(t, np.abs(D), V, 0.5)
    n = np.bincount(t[(t >= 0) & (t < V)], minlength=V)[:, None]
    assert np.all(np.abs(got.cpu().double().numpy() - want) <= (n + 12) * U * size + 2 * U * np.abs(want))
