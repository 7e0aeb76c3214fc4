"""From hidden states to tokens by the framework's own way: the head's logits as a linear_act product, then sampling; for
vocabularies that are multiples of 8, as that product's widths have to be, and for others."""

import os
import sys

import numpy as np
import pytest
import torch

from memory_bounded_linear_gb300 import api
from oracle import token_ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import block_and_head as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def _np(t):
    return t.detach().cpu().double().numpy()


def _model(dt, vocab):
    torch.manual_seed(vocab)
    return ex.TokenModel(72, 200, vocab, device="cuda", dtype={"bf16": torch.bfloat16, "f32": torch.float32}[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [520, 521, 527, 7])
def test_decoding(cuda_lib, vocab, dt):
    """Tokens are those of the distribution of the logits, drawn together and one at a time."""
    m = _model(dt, vocab)
    tokens = torch.randint(0, vocab, (13,), device="cuda")
    logits = m.logits(tokens)
    assert logits.shape == (13, vocab)
    # the product: 72 terms, each rounded to 2^-24 of its size on the way, and the result's own rounding
    h, E = _np(m.hidden(tokens)), _np(m.table)
    limit = 80 * 2.0 ** -24 * (np.abs(h) @ np.abs(E).T) + (2.0 ** -8 if dt == "bf16" else 2.0 ** -24) * np.abs(h @ E.T)
    assert np.all(np.abs(_np(logits) - h @ E.T) <= limit)
    u = torch.rand(13, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    s = dict(temperature=0.7, top_k=40, top_p=0.9)
    together, logprobs = api.lce_sample(logits, u, **s)
    for i in range(13):
        want, lp = token_ref.sample(_np(logits[i]), u[i].item(), float(np.float32(0.7)), 40, float(np.float32(0.9)))
        assert together[i].item() == want and abs(logprobs[i].item() - lp) <= 2.0 ** -20 * max(1.0, abs(lp))
        one, lp = api.lce_sample(logits[i:i + 1], u[i:i + 1], **s)
        assert one.item() == want and lp.item() == logprobs[i].item()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [520, 521])
def test_generate(cuda_lib, vocab, dt):
    """The example's decoding: greedy tokens are the largest logit's, drawn ones those of the same random numbers."""
    m = _model(dt, vocab)
    start = torch.randint(0, vocab, (5,), device="cuda")
    text = m.generate(start, 4, temperature=0.0)
    assert text.shape == (5, 5) and torch.equal(text[:, 0], start)
    for k in range(4):
        assert torch.equal(text[:, k + 1], m.logits(text[:, k].contiguous()).argmax(-1))
    g = torch.Generator(device="cuda").manual_seed(9)
    text = m.generate(start, 3, temperature=0.8, top_k=50, generator=g)
    g.manual_seed(9)
    for k in range(3):
        u = torch.rand(5, generator=g, device="cuda")
        assert torch.equal(text[:, k + 1], api.lce_sample(m.logits(text[:, k].contiguous()), u, temperature=0.8, top_k=50)[0])


def test_example_with_an_odd_vocabulary(cuda_lib):
    losses, norms, text = ex.main(["--tokens", "100", "--width", "64", "--ffn", "136", "--vocab", "333", "--steps", "2",
                                   "--from-tokens"])
    assert np.isfinite(losses).all() and np.isfinite(norms).all()
    assert text.shape == (4, 9) and int(text.min()) >= 0 and int(text.max()) < 333
