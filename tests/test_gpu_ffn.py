"""The feed-forward operators on the GPU against their float64 definitions.

Tolerances (relative Frobenius error unless said otherwise), from the number formats:
* bf16 results of a forward pass: one rounding, at most 2^-9 relative per element, plus fp32 sums
  far below it: 2^-8.  Element by element: 2^-8 of the element plus 2^-8 of the results' rms
  (elements that cancel carry the fp32 sum's error, which is relative to the terms).
* bf16 gradients: the pre-activations' gradient is rounded as an operand (2^-9 of each term) and
  the result again: at most 2^-8 in all where the errors add up; 2^-7.
* fp32: a sum of K products in some order has a random error of about sqrt(K) 2^-24 of the terms'
  norm and a worst one of K 2^-24; at K <= 4096 1e-5 lies between them, and 2e-5 for gradients,
  whose operands carry the same error a second time.
"""

import numpy as np
import pytest
import torch

from memory_bounded_linear_gb300 import api
from oracle import ffn_ref as ref

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
FWD = {"bf16": 2.0 ** -8, "f32": 1e-5}
BWD = {"bf16": 2.0 ** -7, "f32": 2e-5}


def _rand(seed, dt, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(DT[dt])


def _np(t):
    return t.detach().cpu().double().numpy()


def _check(got, want, tol, what=""):
    got = _np(got)
    assert got.shape == want.shape
    assert np.all(np.isfinite(got)), what
    n = np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= tol * n, (what, np.linalg.norm(got - want) / max(n, 1e-300))
    if want.size:
        rms = n / np.sqrt(want.size)
        worst = np.max(np.abs(got - want) / (np.abs(want) + rms))
        assert worst <= 8 * tol, (what, worst)


def _gated_case(dt, N, d, F, act, seed=0):
    x = _rand(seed, dt, N, d)
    wg, wu = (_rand(seed + k, dt, F, d, std=d ** -0.5) for k in (1, 2))
    dh = _rand(seed + 3, dt, N, F)
    h, ws = api.lce_gated_forward(x.cuda(), wg.cuda(), wu.cuda(), activation=act)
    api.lce_check_error(ws)
    dx, dwg, dwu, ws = api.lce_gated_backward(x.cuda(), wg.cuda(), wu.cuda(), dh.cuda(), activation=act)
    api.lce_check_error(ws)
    a = [_np(t) for t in (x, wg, wu)]
    _check(h, ref.gated(*a, act), FWD[dt], "h")
    for got, want, name in zip((dx, dwg, dwu), ref.gated_backward(*a, _np(dh), act), ("dx", "dwg", "dwu")):
        _check(got, want, BWD[dt], name)


def _linear_case(dt, N, di, do, act, bias, residual, seed=0):
    x, w = _rand(seed, dt, N, di), _rand(seed + 1, dt, do, di, std=di ** -0.5)
    b = _rand(seed + 2, dt, do) if bias else None
    r = _rand(seed + 3, dt, N, do) if residual else None
    dy = _rand(seed + 4, dt, N, do)
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    n = lambda t: None if t is None else _np(t)  # noqa: E731
    y, ws = api.lce_linear_forward(c(x), c(w), c(b), c(r), activation=act)
    api.lce_check_error(ws)
    _check(y, ref.linear(n(x), n(w), n(b), n(r), act), FWD[dt], "y")
    dx, dw, db, ws = api.lce_linear_backward(c(x), c(w), c(b), c(dy), activation=act)
    api.lce_check_error(ws)
    want = ref.linear_backward(n(x), n(w), n(b), n(dy), act)
    _check(dx, want[0], BWD[dt], "dx")
    _check(dw, want[1], BWD[dt], "dw")
    assert (db is None) == (b is None)
    if bias:
        _check(db, want[2], BWD[dt], "db")


# one token to several tiles of 256, with the neighbours of 16, 32, 64, 128 and 256
TOKENS = [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 48, 63, 64, 65, 100, 127, 128, 129, 200, 255, 256, 257, 520]


@pytest.mark.parametrize("N", TOKENS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gated_over_token_counts(cuda_lib, dt, N):
    _gated_case(dt, N, 200, 264, "silu", seed=N)


@pytest.mark.parametrize("N", TOKENS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_linear_over_token_counts(cuda_lib, dt, N):
    _linear_case(dt, N, 264, 200, "none", True, True, seed=N)


@pytest.mark.parametrize("act", ref.ACTIVATIONS)
@pytest.mark.parametrize("N", [3, 300])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_activations(cuda_lib, dt, N, act):
    _gated_case(dt, N, 64, 136, act, seed=11)
    _linear_case(dt, N, 136, 72, act, True, False, seed=12)


# widths: the smallest row, under one k-block, ends inside a k-block or a tile, several tiles
WIDTHS = [(8, 8), (8, 136), (136, 8), (56, 64), (64, 128), (72, 120), (128, 1000), (1032, 256),
          (520, 328), (4096, 24), (24, 2056)]


@pytest.mark.parametrize("N", [1, 5, 40, 130, 257])
@pytest.mark.parametrize("a,b", WIDTHS)
def test_widths_bf16(cuda_lib, a, b, N):
    _gated_case("bf16", N, a, b, "gelu", seed=a + b)
    _linear_case("bf16", N, a, b, "silu", True, True, seed=a + b)
    _linear_case("bf16", N, a, b, "none", False, False, seed=a + b)


@pytest.mark.parametrize("N", [1, 40, 257])
@pytest.mark.parametrize("a,b", [(4, 4), (4, 132), (132, 12), (60, 68), (1028, 260), (2052, 20)])
def test_widths_f32(cuda_lib, a, b, N):
    _gated_case("f32", N, a, b, "gelu_tanh", seed=a + b)
    _linear_case("f32", N, a, b, "gelu", True, True, seed=a + b)
    _linear_case("f32", N, a, b, "none", True, False, seed=a + b)


def _act64(z, name):
    if name == "none":
        return z
    if name == "silu":
        return z * torch.sigmoid(z)
    return 0.5 * z * torch.erfc(-z * 0.5 ** 0.5)


def _close(got, want, tol, what):
    assert torch.isfinite(got).all(), what
    err = (got.double() - want).norm() / want.norm()
    assert err <= tol, (what, err.item())


# tokens, widths: sums over many tokens beside short ones, many tiles (taken as tickets), operands whose
# rows are copied, long sums of few and of many tokens, every kind at sizes of a real block
# fp32 forward passes on both sides of the choice between dot products and tiles: one to eight warps per
# sum, ragged token tiles and feature groups, K that ends inside a warp's step, the largest N
F32_FORWARD = [(3, 132, 8196), (8, 2048, 2052), (13, 1028, 2004), (21, 516, 1028), (45, 4, 4), (48, 2052, 260),
               (49, 260, 1004), (77, 6004, 132), (333, 1028, 1004), (301, 516, 1004), (4096, 36, 20),
               (4097, 36, 20), (1000, 260, 516), (2, 1028, 4100)]


@pytest.mark.parametrize("N,d,F", F32_FORWARD)
def test_f32_forward(cuda_lib, N, d, F):
    """Against plain products in float64 on the GPU, into a padded result whose padding stays."""
    g = torch.Generator(device="cuda").manual_seed(N + d)
    x, w, wu, b, r = (torch.randn(*s, generator=g, device="cuda") * k for s, k in (
        ((N, d), 1.0), ((F, d), d ** -0.5), ((F, d), d ** -0.5), ((F,), 1.0), ((N, F), 1.0)))
    z, u = x.double() @ w.double().t(), x.double() @ wu.double().t()
    for act in ("gelu", "none"):
        out = torch.full((N, F + 4), 7.0, device="cuda")
        y, ws = api.lce_linear_forward(x, w, b, r, activation=act, out=out[:, :F])
        api.lce_check_error(ws)
        _close(y, _act64(z + b.double(), act) + r.double(), FWD["f32"], "y " + act)
        assert torch.all(out[:, F:] == 7.0)
    h, ws = api.lce_gated_forward(x, w, wu, activation="silu")
    api.lce_check_error(ws)
    _close(h, _act64(z, "silu") * u, FWD["f32"], "h")


LARGE = [(16384, 128, 264, "bf16"), (8192, 132, 260, "f32"), (20000, 64, 5128, "bf16"), (4096, 1024, 4096, "bf16"),
         (2600, 1032, 2600, "bf16"), (2600, 520, 2616, "bf16"), (40, 16384, 520, "bf16"), (7, 12288, 1024, "f32"),
         (150, 8192, 2048, "bf16"), (150, 1024, 11008, "bf16"), (600, 9216, 520, "bf16"), (500, 4096, 516, "f32"),
         (1000, 2048, 8192, "bf16")]


@pytest.mark.parametrize("N,d,F,dt", LARGE)
def test_large_shapes(cuda_lib, N, d, F, dt):
    """Against plain products in float64 on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(N + d)
    rand = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(DT[dt])  # noqa: E731
    x, wg, wu, dh, b = rand(N, d), rand(F, d, std=d ** -0.5), rand(F, d, std=d ** -0.5), rand(N, F), rand(F)
    X, G, U, D = (t.double().requires_grad_() for t in (x, wg, wu, b))
    want = _act64(X @ G.t(), "silu") * (X @ U.t())
    h, _ = api.lce_gated_forward(x, wg, wu)
    _close(h, want.detach(), FWD[dt], "h")
    grads = torch.autograd.grad((want * dh.double()).sum(), (X, G, U))
    for name, a, w in zip(("dx", "dwg", "dwu"), api.lce_gated_backward(x, wg, wu, dh), grads):
        _close(a, w, BWD[dt], name)
    del want, grads
    for act in ("gelu", "none"):
        want = _act64(X @ G.t() + D, act)
        y, _ = api.lce_linear_forward(x, wg, b, dh, activation=act)
        _close(y, want.detach() + dh.double(), FWD[dt], "y")
        grads = torch.autograd.grad((want * dh.double()).sum(), (X, G, D))
        for name, a, w in zip(("dx", "dw", "db"), api.lce_linear_backward(x, wg, b, dh, activation=act), grads):
            _close(a, w, BWD[dt], name)


@pytest.mark.parametrize("N,d,F", [(150, 128, 20_000), (150, 1024, 11_008), (100, 136, 30_000), (700, 8, 40_000)])
def test_short_sums_store_every_tile(cuda_lib, N, d, F):
    """Weight gradients of few tokens: many tiles of short sums whose results leave as fast as the
    boxes they leave through come free; a box written too early shows as wrong values in some of
    many rounds."""
    x, dy = _rand(1, "bf16", N, d).cuda(), _rand(2, "bf16", N, F).cuda()
    w = _rand(3, "bf16", F, d, std=d ** -0.5).cuda()
    want = dy.double().t() @ x.double()
    first = None
    for _ in range(20):
        dw = api.lce_linear_backward(x, w, None, dy, parts="dw")[1]
        if first is None:
            first = dw
            assert ((dw.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-3 * N ** 0.5).all()
        assert torch.equal(dw, first)


def test_past_32_bit_offsets(cuda_lib):
    """Results of more than 2^31 elements: the first and last rows, and sums over all of them."""
    N, d, F = 70_000, 64, 32_768
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
    x, wg, wu = rand(N, d), rand(F, d, std=0.125), rand(F, d, std=0.125)
    rows = torch.tensor([0, 1, N // 2, N - 257, N - 2, N - 1], device="cuda")
    cols = torch.tensor([0, 5, F // 2, F - 1], device="cuda")
    out = torch.full((N, F), 3.0, dtype=torch.bfloat16, device="cuda")
    api.lce_gated_forward(x, wg, wu, out=out)
    X, G, U = x.double(), wg.double(), wu.double()
    _close(out[rows], _act64(X[rows] @ G.t(), "silu") * (X[rows] @ U.t()), FWD["bf16"], "h")
    dx, dwg, dwu, _ = api.lce_gated_backward(x, wg, wu, out)     # dH = H
    o = out[rows].double()
    z, u = X[rows] @ G.t(), X[rows] @ U.t()
    s = torch.sigmoid(z)
    _close(dx[rows], (o * u * (s + z * s * (1 - s))) @ G + (o * z * s) @ U, BWD["bf16"], "dx")
    o = out[:, cols].double()
    z, u = X @ G[cols].t(), X @ U[cols].t()
    s = torch.sigmoid(z)
    _close(dwg[cols], (o * u * (s + z * s * (1 - s))).t() @ X, BWD["bf16"], "dwg")
    _close(dwu[cols], (o * z * s).t() @ X, BWD["bf16"], "dwu")
    r = torch.full_like(out, 0.5)
    api.lce_linear_forward(x, wg, None, r, out=r)                # in place, past 2^31
    _close(r[rows], X[rows] @ G.t() + 0.5, FWD["bf16"], "y")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [6, 300])
def test_row_strides_and_in_place_residual(cuda_lib, dt, N):
    di, do = 72, 136
    wide = _rand(1, dt, N, 3 * di).cuda()
    x = wide[:, di:2 * di]
    w, b = _rand(2, dt, do, di).cuda(), _rand(3, dt, do).cuda()
    rw = _rand(4, dt, N, do + 40).cuda()
    r = rw[:, 8:8 + do]
    ow = torch.full((N, do + 64), 7.0, dtype=DT[dt], device="cuda")
    out = ow[:, 16:16 + do]
    want = ref.linear(_np(x), _np(w), _np(b), _np(r), "relu")
    y, _ = api.lce_linear_forward(x, w, b, r, activation="relu", out=out)
    assert y is out
    _check(y, want, FWD[dt])
    assert torch.all(ow[:, :16] == 7) and torch.all(ow[:, 16 + do:] == 7)   # nothing beside the rows
    before = rw.clone()
    y, _ = api.lce_linear_forward(x, w, b, r, activation="relu", out=r)     # added in place
    _check(y, want, FWD[dt])
    assert torch.equal(rw[:, :8], before[:, :8]) and torch.equal(rw[:, 8 + do:], before[:, 8 + do:])
    dyw = _rand(5, dt, N, do + 8).cuda()
    dy = dyw[:, :do]
    got = api.lce_linear_backward(x, w, b, dy, activation="relu")
    for g, t in zip(got, ref.linear_backward(_np(x), _np(w), _np(b), _np(dy), "relu")):
        _check(g, t, BWD[dt])
    wu = _rand(6, dt, do, di).cuda()
    h, _ = api.lce_gated_forward(x, w, wu, out=out)
    _check(h, ref.gated(_np(x), _np(w), _np(wu)), FWD[dt])
    assert torch.all(ow[:, :16] == 7) and torch.all(ow[:, 16 + do:] == 7)
    got = api.lce_gated_backward(x, w, wu, dy)
    for g, t in zip(got, ref.gated_backward(_np(x), _np(w), _np(wu), _np(dy))):
        _check(g, t, BWD[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_no_tokens(cuda_lib, dt):
    x = torch.empty(0, 64, dtype=DT[dt], device="cuda")
    w = _rand(1, dt, 96, 64).cuda()
    b = _rand(2, dt, 96).cuda()
    dy = torch.empty(0, 96, dtype=DT[dt], device="cuda")
    assert api.lce_linear_forward(x, w, b)[0].shape == (0, 96)
    assert api.lce_gated_forward(x, w, w)[0].shape == (0, 96)
    dx, dw, db, _ = api.lce_linear_backward(x, w, b, dy, activation="gelu")
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    dx, dwg, dwu, _ = api.lce_gated_backward(x, w, w, dy)
    assert dx.shape == (0, 64) and not dwg.any() and not dwu.any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [5, 300])
def test_parts_equal_the_whole(cuda_lib, dt, N):
    x, w, wu = _rand(1, dt, N, 136).cuda(), _rand(2, dt, 200, 136).cuda(), _rand(3, dt, 200, 136).cuda()
    b, dy = _rand(4, dt, 200).cuda(), _rand(5, dt, N, 200).cuda()
    both = api.lce_linear_backward(x, w, b, dy, activation="gelu")
    dx = api.lce_linear_backward(x, w, b, dy, activation="gelu", parts="dx")
    dw = api.lce_linear_backward(x, w, b, dy, activation="gelu", parts="dw")
    assert dx[1] is None and dx[2] is None and dw[0] is None
    assert torch.equal(dx[0], both[0]) and torch.equal(dw[1], both[1]) and torch.equal(dw[2], both[2])
    both = api.lce_gated_backward(x, w, wu, dy)
    dx, dw = (api.lce_gated_backward(x, w, wu, dy, parts=p) for p in ("dx", "dw"))
    assert torch.equal(dx[0], both[0])
    assert torch.equal(dw[1], both[1]) and torch.equal(dw[2], both[2])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [4, 1000])
def test_results_repeat_bit_for_bit(cuda_lib, dt, N):
    x, w, wu = _rand(1, dt, N, 520).cuda(), _rand(2, dt, 776, 520).cuda(), _rand(3, dt, 776, 520).cuda()
    b, dy = _rand(4, dt, 776).cuda(), _rand(5, dt, N, 776).cuda()

    def everything():
        return [api.lce_gated_forward(x, w, wu)[0], *api.lce_gated_backward(x, w, wu, dy)[:3],
                api.lce_linear_forward(x, w, b, dy, activation="gelu")[0],
                *api.lce_linear_backward(x, w, b, dy, activation="gelu")[:3]]
    first = everything()
    for _ in range(3):
        assert all(torch.equal(a, c) for a, c in zip(first, everything()))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N", [9, 270])
def test_rows_do_not_mix(cuda_lib, dt, N):
    """A NaN, an inf or a huge value in one token's row reaches that row alone; one in a weight
    row reaches that output column alone."""
    x, w, wu = _rand(1, dt, N, 136).cuda(), _rand(2, dt, 200, 136).cuda(), _rand(3, dt, 200, 136).cuda()
    clean = [api.lce_linear_forward(x, w)[0], api.lce_gated_forward(x, w, wu)[0]]
    bad = x.clone()
    bad[3, 7], bad[5, 0] = float("nan"), float("inf")
    for k, got in enumerate([api.lce_linear_forward(bad, w)[0], api.lce_gated_forward(bad, w, wu)[0]]):
        assert not torch.isfinite(got[3]).any() and not torch.isfinite(got[5]).all()
        keep = [i for i in range(N) if i not in (3, 5)]
        assert torch.equal(got[keep], clean[k][keep])
    wbad = w.clone()
    wbad[11, 2] = float("nan")
    for k, got in enumerate([api.lce_linear_forward(x, wbad)[0], api.lce_gated_forward(x, wbad, wu)[0]]):
        assert torch.isnan(got[:, 11]).all()
        cols = [i for i in range(200) if i != 11]
        assert torch.equal(got[:, cols], clean[k][:, cols])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_relu_masks_what_is_not_finite(cuda_lib, dt):
    """An inf or NaN of the outgoing gradient where the ReLU is 0 does not reach the gradients."""
    N, d, out = 70, 72, 136
    x = torch.ones(N, d, dtype=DT[dt])
    w = _rand(1, dt, out, d).abs()
    w[::3] *= -1                                     # every third output is below zero in all rows
    wu, dy = _rand(2, dt, out, d, std=d ** -0.5), _rand(3, dt, N, out)
    bad = dy.clone()
    bad[0, 0], bad[5, 3], bad[69, 135] = float("nan"), float("inf"), float("-inf")
    args = x.cuda(), w.cuda()
    for clean, got in zip(api.lce_linear_backward(*args, None, dy.cuda(), activation="relu")[:2],
                          api.lce_linear_backward(*args, None, bad.cuda(), activation="relu")[:2]):
        assert torch.isfinite(got).all() and torch.equal(got, clean)
    clean = api.lce_gated_backward(*args, wu.cuda(), dy.cuda(), activation="relu")[1]
    got = api.lce_gated_backward(*args, wu.cuda(), bad.cuda(), activation="relu")[1]
    assert torch.isfinite(got).all() and torch.equal(got, clean)


def test_large_magnitudes_of_the_activations(cuda_lib):
    """Pre-activations far outside the exponential's range: results stay finite and exact limits."""
    z = torch.tensor([-3e38, -1e30, -200.0, -90.0, -88.0, 0.0, 88.0, 90.0, 200.0, 1e30], dtype=torch.float32)
    for dt in ("bf16", "f32"):
        x = torch.zeros(z.numel(), 8, dtype=DT[dt])
        x[:, 0] = z.to(DT[dt])
        w = torch.zeros(8, 8, dtype=DT[dt])
        w[0, 0] = 1.0
        for act in ("relu", "silu", "gelu", "gelu_tanh"):
            y = api.lce_linear_forward(x.cuda(), w.cuda(), activation=act)[0][:, 0].cpu().double()
            want = torch.where(z > 0, x[:, 0].double(), torch.zeros(1, dtype=torch.float64))
            assert torch.isfinite(y).all(), (dt, act)
            assert torch.all((y - want).abs() <= 1e-2 * want.abs() + 1e-30), (dt, act, y)
            dx = api.lce_linear_backward(x.cuda(), w.cuda(), None, w[0].repeat(z.numel(), 1).cuda(),
                                         activation=act)[0][:, 0].cpu().double()
            slope = torch.where(z > 0, 1.0, 0.0).double()
            slope[5] = 0.0 if act == "relu" else 0.5
            assert torch.all((dx - slope).abs() <= 1e-2), (dt, act, dx)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_autograd(cuda_lib, dt):
    """The autograd functions: leading dimensions, an expanded outgoing gradient, gradients only
    where they are asked for."""
    x = _rand(1, dt, 3, 7, 64).cuda().requires_grad_()
    wg, wu = (_rand(k, dt, 96, 64, std=0.125).cuda().requires_grad_() for k in (2, 3))
    wd, b = _rand(4, dt, 64, 96, std=0.1).cuda().requires_grad_(), _rand(5, dt, 64).cuda().requires_grad_()
    h = api.gated_linear(x, wg, wu, "silu")
    y = api.linear_act(h, wd, b, x, activation="gelu")
    assert y.shape == x.shape
    y.sum().backward()                              # a gradient with no strides of its own
    X, G, U, D, B = (_np(t) for t in (x.reshape(-1, 64), wg, wu, wd, b))
    H = _np(h.reshape(-1, 96))                      # as rounded by the first operator
    one = np.ones((21, 64))
    dh, dwd, db = ref.linear_backward(H, D, B, one, "gelu")
    _check(wd.grad, dwd, BWD[dt], "wd")
    _check(b.grad, db, BWD[dt], "b")
    dx, dwg, dwu = ref.gated_backward(X, G, U, dh, "silu")
    # dh is rounded once more on its way to the first operator
    _check(wg.grad, dwg, 2 * BWD[dt], "wg")
    _check(wu.grad, dwu, 2 * BWD[dt], "wu")
    _check(x.grad.reshape(-1, 64), dx + one, 2 * BWD[dt], "x")
    frozen = api.gated_linear(x.detach(), wg.detach(), wu, "silu")
    assert frozen.requires_grad
    g = torch.autograd.grad(frozen.sum(), wu)[0]
    assert g.shape == wu.shape
    assert not api.linear_act(x.detach(), wg.detach()).requires_grad


@pytest.mark.parametrize("which", ["linear", "gated"])
def test_gradient_against_differences(cuda_lib, which):
    """fp32: the directional derivative of sum(out * dy) along a random direction, by central
    differences of the float64 definition at a step of 1e-4 (error about 1e-8 of the value), against
    the gradient's inner product with the direction (fp32 gradient: 2e-5 of the norms)."""
    x, wg, wu = _rand(1, "f32", 40, 36), _rand(2, "f32", 52, 36, std=0.2), _rand(3, "f32", 52, 36, std=0.2)
    b, dy = _rand(4, "f32", 52), _rand(5, "f32", 40, 52)
    dirs = [np.random.RandomState(9 + k).randn(*t.shape) for k, t in enumerate((x, wg, wu))]
    X, G, U, B, DY = (_np(t) for t in (x, wg, wu, b, dy))
    if which == "gated":
        f = lambda s: np.sum(ref.gated(X + s * dirs[0], G + s * dirs[1], U + s * dirs[2], "silu") * DY)  # noqa: E731
        grads = api.lce_gated_backward(x.cuda(), wg.cuda(), wu.cuda(), dy.cuda())[:3]
    else:
        f = lambda s: np.sum(ref.linear(X + s * dirs[0], G + s * dirs[1], B, None, "gelu") * DY)  # noqa: E731
        grads = api.lce_linear_backward(x.cuda(), wg.cuda(), b.cuda(), dy.cuda(), activation="gelu")[:2]
    want = (f(1e-4) - f(-1e-4)) / 2e-4
    got = sum(np.sum(_np(g) * v) for g, v in zip(grads, dirs))
    scale = sum(np.linalg.norm(_np(g)) * np.linalg.norm(v) for g, v in zip(grads, dirs))
    assert abs(got - want) <= 2e-5 * scale


def test_stream_and_graph(cuda_lib):
    """On a stream other than the current one, and captured in a graph and replayed on new inputs."""
    x, w, wu = _rand(1, "bf16", 300, 136).cuda(), _rand(2, "bf16", 200, 136).cuda(), _rand(3, "bf16", 200, 136).cuda()
    dy = _rand(4, "bf16", 300, 200).cuda()
    want = [api.lce_gated_forward(x, w, wu)[0], *api.lce_gated_backward(x, w, wu, dy)[:3]]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [api.lce_gated_forward(x, w, wu, stream=s)[0], *api.lce_gated_backward(x, w, wu, dy, stream=s)[:3]]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    few = x[:3].clone()
    with torch.cuda.stream(s):
        api.lce_gated_forward(few, w, wu)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = [api.lce_gated_forward(x, w, wu)[0], *api.lce_gated_backward(x, w, wu, dy)[:3],
                   api.lce_gated_forward(few, w, wu)[0]]
    x2 = _rand(7, "bf16", 300, 136).cuda()
    x.copy_(x2)
    few.copy_(x2[:3])
    g.replay()
    torch.cuda.synchronize()
    want = [api.lce_gated_forward(x, w, wu)[0], *api.lce_gated_backward(x, w, wu, dy)[:3],
            api.lce_gated_forward(few, w, wu)[0]]
    assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("captured", [False, True])
def test_order_with_other_work_on_the_stream(cuda_lib, captured):
    """Calls read what a memset, a copy and other kernels before them wrote, and what follows them (a
    copy, an in-place kernel, the same call again) sees their results: round after round, with inputs
    that change, on one stream."""
    N, d, F = 3, 520, 1032
    x, xs = torch.zeros(N, d, dtype=torch.bfloat16, device="cuda"), _rand(1, "bf16", 6, N, d).cuda()
    w, wu = _rand(2, "bf16", F, d, std=0.04).cuda(), _rand(3, "bf16", F, d, std=0.04).cuda()
    wd, b = _rand(4, "bf16", d, F, std=0.03).cuda(), _rand(5, "bf16", d).cuda()
    h = torch.zeros(N, F, dtype=torch.bfloat16, device="cuda")
    results = torch.zeros(6, N, d, dtype=torch.bfloat16, device="cuda")
    grads = [torch.zeros(N, d, device="cuda")]

    def rounds():
        for k in range(6):
            x.zero_()
            x.copy_(xs[k])
            h.zero_()
            api.lce_gated_forward(x, w, wu, out=h)
            api.lce_linear_forward(h, wd, b, x, out=x)
            x.mul_(0.5)
            api.lce_gated_forward(x, w, wu, out=h)
            api.lce_linear_forward(h, wd, b, x, out=results[k])
            grads[0].copy_(results[k])
            api.lce_clip_grad_norm(grads, 1.0)
            results[k].copy_(grads[0])
    if captured:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            rounds()
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            rounds()
        xs.mul_(1.5)
        for _ in range(3):
            results.fill_(7.0)
            g.replay()
    else:
        for _ in range(3):
            rounds()
    torch.cuda.synchronize()
    for k in range(6):
        step = xs[k].clone()
        for i in range(2):
            torch.cuda.synchronize()
            hh = api.lce_gated_forward(step, w, wu)[0]
            torch.cuda.synchronize()
            step = api.lce_linear_forward(hh, wd, b, step)[0]
            torch.cuda.synchronize()
            if i == 0:
                step.mul_(0.5)
        gr = step.float()
        torch.cuda.synchronize()
        want = api.lce_clip_grad_norm([gr], 1.0)[1][0].bfloat16()
        assert torch.equal(results[k], want), k


def test_refusals_on_the_gpu(cuda_lib):
    x, w = torch.zeros(4, 64, device="cuda"), torch.zeros(96, 64, device="cuda")
    with pytest.raises(TypeError):
        api.lce_linear_forward(x.half(), w.half())
    with pytest.raises(TypeError):
        api.lce_linear_forward(x, w.bfloat16())
    with pytest.raises(ValueError):
        api.lce_linear_forward(x, w, torch.zeros(95, device="cuda"))
    with pytest.raises(ValueError):
        api.lce_linear_forward(x, w.t().contiguous().t())
    with pytest.raises(ValueError):
        api.lce_linear_forward(x[:, :1].expand(4, 64), w)
    with pytest.raises(ValueError):
        api.lce_linear_forward(x, w, residual=torch.zeros(1, 96, device="cuda").expand(4, 96))
    with pytest.raises(ValueError):
        api.lce_gated_forward(x, w, w[:, :32])
    with pytest.raises(ValueError, match="activation"):
        api.lce_gated_forward(x, w, w, activation="tanh")
    with pytest.raises(ValueError, match="parts"):
        api.lce_gated_backward(x, w, w, torch.zeros(4, 96, device="cuda"), parts="dh")
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        api.lce_linear_forward(x, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(RuntimeError, match="INVALID_ARG"):
        api.lce_linear_forward(x, w, out=x[:, :64] if w.shape[0] == 64 else torch.zeros(4, 97, device="cuda")[:, 1:])
    with pytest.raises(RuntimeError, match="SHAPE"):
        api.lce_linear_forward(x[:, :62].contiguous(), w[:, :62].contiguous())
