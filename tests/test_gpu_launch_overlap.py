"""Launches that begin while the one before ends: clipping directly behind the kernels that write the
gradients, round after round in place, and calls on two streams at once."""

import pytest
import torch

from memory_bounded_linear_gb300 import api

pytestmark = pytest.mark.gpu


def _rand(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,d,F", [(40, 264, 520), (700, 512, 1024)])
def test_clipping_behind_the_backward_pass(cuda_lib, N, d, F, dtype):
    """The gradients, clipped in place three times with nothing between the launches, against the same
    calls with a synchronisation between any two."""
    xs = _rand(1, 8, N, d, dtype=dtype)
    w, b, dy = _rand(2, F, d, std=0.05, dtype=dtype), _rand(3, F, dtype=dtype), _rand(4, N, F, dtype=dtype)

    def rounds(pause):
        out = []
        for x in xs:
            g = list(api.lce_linear_backward(x, w, b, dy, activation="silu")[:3])
            pause()
            for k in range(3):
                out.append(api.lce_clip_grad_norm(g, 1.0 / (k + 1))[0])
                pause()
            out += [t.clone() for t in g]
            pause()
        return out
    want = rounds(torch.cuda.synchronize)
    for _ in range(5):
        assert all(torch.equal(a, c) for a, c in zip(rounds(lambda: None), want))


def test_many_unaligned_arrays_in_place(cuda_lib):
    """More arrays than one table, at every alignment, clipped again and again: each round sees what the
    one before wrote."""
    sizes = [(k * 37) % 501 + 1 for k in range(1300)]
    flat = _rand(5, sum(sizes) + 7, dtype=torch.float32)
    begin = [7 + sum(sizes[:k]) for k in range(len(sizes))]

    def rounds(pause):
        buf = flat.clone()
        grads = [buf[i:i + n] for i, n in zip(begin, sizes)]
        totals = []
        for k in range(6):
            pause()
            totals.append(api.lce_clip_grad_norm(grads, 100.0 * 0.7 ** k)[0])
        pause()
        return [torch.stack(totals), buf]
    want = rounds(torch.cuda.synchronize)
    expected = flat[7:].double().norm().item()
    for k, t in enumerate(want[0].tolist()):
        assert abs(t - expected) <= 1e-5 * expected
        expected = min(expected, 100.0 * 0.7 ** k)
    assert torch.equal(want[1][:7], flat[:7])
    for _ in range(5):
        assert all(torch.equal(a, c) for a, c in zip(rounds(lambda: None), want))


def test_two_streams(cuda_lib):
    """Calls of every kind on two streams at once, each with its own workspaces: the same bits as alone."""
    def everything(seed, N):
        x, w, wu = _rand(seed, N, 520), _rand(seed + 1, 1032, 520, std=0.04), _rand(seed + 2, 1032, 520, std=0.04)
        dy, xf, wf = _rand(seed + 3, N, 1032), _rand(seed + 4, 90, 260, dtype=torch.float32), \
            _rand(seed + 5, 516, 260, dtype=torch.float32)
        dyf = _rand(seed + 6, 90, 516, dtype=torch.float32)

        def go():
            r = [api.lce_gated_forward(x[:3], w, wu)[0], api.lce_gated_forward(x[:40], w, wu)[0],
                 api.lce_gated_forward(x, w, wu)[0], *api.lce_gated_backward(x, w, wu, dy)[:3],
                 *api.lce_linear_backward(x, w, None, dy, activation="gelu")[:2],
                 api.lce_linear_forward(xf, wf)[0], *api.lce_gated_backward(xf, wf, wf, dyf)[:3]]
            api.lce_clip_grad_norm(r, 1.0)
            return r
        return go
    calls = [everything(10, 300), everything(30, 700)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        got = [[], []]
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k] = calls[k]()
        torch.cuda.synchronize()
        for a, c in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, c))
