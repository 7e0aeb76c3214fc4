"""Global gradient norm and clipping against float64.

Tolerances: the total is a sum of non-negative fp32 squares (2^-24 each) over at most 64 values in
fp32 (63 roundings, worst 2^-18, random about 2^-21) and beyond that in fp64, then one rounding:
2^-20 relative (half the sum's error reaches the root).  Scaled values: c in fp32 (total's error and two roundings) times
g, one rounding to the result's type: 2^-19 relative for float32, 2^-8 for bfloat16."""

import numpy as np
import pytest
import torch

from memory_bounded_linear_gb300 import api
from oracle import ffn_ref as ref

pytestmark = pytest.mark.gpu
TOTAL = 2.0 ** -20
SCALED = {torch.float32: 2.0 ** -19, torch.bfloat16: 2.0 ** -8}


def _grads(sizes, seed=0, std=1.0):
    """Alternating types, bfloat16 first."""
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std).to(torch.bfloat16 if k % 2 == 0 else torch.float32).cuda()
            for k, n in enumerate(sizes)]


def _np(ts):
    return [t.detach().cpu().double().numpy() for t in ts]


def _check(out, want, dtypes):
    for o, w, dt in zip(out, want, dtypes):
        o = o.detach().cpu().double().numpy()
        # values below the smallest normal of their type lose bits: allow that much absolutely
        assert np.all(np.abs(o - w) <= SCALED[dt] * np.abs(w) + 2e-38)


SIZES = [[1], [1, 1], [3, 0, 5], [255, 256, 257], [16383, 16384, 16385], [7, 100_003, 1, 65_537, 12],
         [0, 0, 9], [2_000_001, 3], [1 << 22]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("norm", ["l2", "inf"])
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_clip(cuda_lib, sizes, norm, max_norm):
    grads = _grads(sizes, seed=len(sizes))
    total, want = ref.clip(_np(grads), max_norm, norm)
    got, _ = api.lce_grad_norm(grads, norm=norm)
    assert abs(got.item() - total) <= TOTAL * total
    kept = [t.clone() for t in grads]
    out = [torch.full_like(t, 3.0) for t in grads]
    t2, o2, _ = api.lce_clip_grad_norm(grads, max_norm, norm=norm, out=out)
    assert t2.item() == got.item() and all(a is b for a, b in zip(o2, out))
    _check(out, want, [t.dtype for t in grads])
    assert all(torch.equal(a, b) for a, b in zip(grads, kept))        # the inputs stay
    t3, o3, _ = api.lce_clip_grad_norm(grads, max_norm, norm=norm)
    assert t3.item() == got.item() and all(a is b for a, b in zip(o3, grads))
    assert all(torch.equal(a, b) for a, b in zip(grads, out))         # in place: the same values


def test_unaligned_and_offset_views(cuda_lib):
    """Slices of a flat buffer at every offset of 16 bytes; values beside them stay."""
    flat32 = torch.randn(40_000, device="cuda")
    flat16 = torch.randn(40_000, device="cuda").bfloat16()
    for off in range(0, 9):
        for out_off in (off, off + 1):
            grads = [flat32[off:off + 9_001], flat16[off:off + 17_003], flat32[20_000 + off:20_003 + off]]
            bufs = [torch.full((t.numel() + 32,), 5.0, dtype=t.dtype, device="cuda") for t in grads]
            out = [b[out_off:out_off + t.numel()] for b, t in zip(bufs, grads)]
            total, want = ref.clip(_np(grads), 1.0)
            got, _, _ = api.lce_clip_grad_norm(grads, 1.0, out=out)
            assert abs(got.item() - total) <= TOTAL * total
            _check(out, want, [t.dtype for t in grads])
            for b, t in zip(bufs, grads):
                assert torch.all(b[:out_off] == 5) and torch.all(b[out_off + t.numel():] == 5)


def test_many_tensors(cuda_lib):
    """More arrays than one launch's table holds."""
    grads = _grads([(k * 37) % 501 for k in range(1300)])
    total, want = ref.clip(_np(grads), 2.0)
    got, out, _ = api.lce_clip_grad_norm(grads, 2.0)
    assert abs(got.item() - total) <= TOTAL * total
    _check(out, want, [t.dtype for t in grads])


def test_strided_gradients(cuda_lib):
    """A dense transposed gradient is taken in the order of its memory; one with gaps is refused."""
    a = torch.randn(33, 70, device="cuda")
    t = a.t()
    total, want = ref.clip(_np([t]), 1.0)
    got, out, _ = api.lce_clip_grad_norm([t], 1.0)
    assert abs(got.item() - total) <= TOTAL * total
    _check(out, want, [t.dtype])
    with pytest.raises(ValueError, match="dense"):
        api.lce_grad_norm([a[:, :5]])
    with pytest.raises(ValueError, match="dense"):
        api.lce_grad_norm([a[:1].expand(4, 70)])
    with pytest.raises(TypeError):
        api.lce_grad_norm([a.half()])
    with pytest.raises(ValueError, match="strides"):
        api.lce_clip_grad_norm([t], 1.0, out=[torch.empty(70, 33, device="cuda")])


def test_non_finite(cuda_lib):
    for bad in (float("nan"), float("inf"), float("-inf")):
        for dt in (torch.float32, torch.bfloat16):
            for norm in ("l2", "inf"):
                g = [torch.ones(50_000, device="cuda"), torch.ones(7, device="cuda", dtype=dt)]
                g[1][3] = bad
                total, out, _ = api.lce_clip_grad_norm(g, 1.0, norm=norm, out=[torch.empty_like(t) for t in g])
                if bad != bad:
                    assert torch.isnan(total) and torch.isnan(out[0]).all() and torch.isnan(out[1]).all()
                else:
                    assert total.item() == float("inf")
                    assert not out[0].any() and torch.isnan(out[1][3]) and out[1][2].item() == 0


def test_extreme_magnitudes(cuda_lib):
    g = [torch.full((1000,), 3e38, device="cuda"), torch.full((3,), -1e-40, device="cuda")]
    assert api.lce_grad_norm(g, norm="inf")[0].item() == g[0][0].item()
    assert api.lce_grad_norm(g)[0].item() == float("inf")
    z = [torch.zeros(100, device="cuda")]
    total, out, _ = api.lce_clip_grad_norm(z, 0.0)
    assert total.item() == 0.0 and not out[0].any()
    total, out, _ = api.lce_clip_grad_norm([torch.ones(100, device="cuda")], 0.0)
    assert total.item() == 10.0 and not out[0].any()


def test_repeatable_and_captured(cuda_lib):
    grads = _grads([300_001, 5, 77_777])
    totals = {api.lce_grad_norm(grads)[0].item() for _ in range(5)}
    assert len(totals) == 1
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = [torch.empty_like(t) for t in grads]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        total, _, _ = api.lce_clip_grad_norm(grads, 1.0, out=out)
    for t in grads:
        t.mul_(2.0)
    g.replay()
    torch.cuda.synchronize()
    want_total, want = ref.clip(_np(grads), 1.0)
    assert abs(total.item() - want_total) <= TOTAL * want_total
    _check(out, want, [t.dtype for t in grads])


def test_parameters(cuda_lib):
    p = [torch.nn.Parameter(torch.randn(5, 7, device="cuda")), torch.nn.Parameter(torch.zeros(3, device="cuda"))]
    (p[0] * 10).sum().backward()
    total = api.clip_grad_norm_(p, 1.0)
    assert abs(total.item() - 10 * 35 ** 0.5) <= 1e-4
    assert abs(p[0].grad.norm().item() - 1.0) <= 1e-4 and p[1].grad is None


def test_past_32_bit_offsets(cuda_lib):
    """An array of more than 2^31 elements: its last values take part and are scaled."""
    n = (1 << 31) + 40_000
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-3:] = 4.0
    g[5] = 4.0
    total, out, _ = api.lce_clip_grad_norm([g], 4.0)
    assert total.item() == 8.0
    assert torch.all(out[0][-3:] == 2.0) and out[0][5].item() == 2.0 and out[0][6].item() == 0.0
