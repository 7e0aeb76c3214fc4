"""Refusals of the feed-forward and clipping entry points, no GPU needed: every call below returns
from the checks of its arguments; none reaches the CUDA runtime."""

import ctypes
import os

import pytest
import torch

from memory_bounded_linear_gb300 import _lib, api


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from memory_bounded_linear_gb300.csrc import build
        build.build()
    return _lib.load()


class _Buf:
    """Host memory that stands in for device pointers; the checks fail before any access."""

    def __init__(self, n=1 << 16):
        self.raw = ctypes.create_string_buffer(n + 64)
        self.addr = (ctypes.addressof(self.raw) + 63) // 64 * 64


BUF = _Buf()
P = BUF.addr
BIG = 1 << 40


def test_names(lib):
    names = {lib.lce_kernel_name(i).decode() for i in range(11, 20)}
    assert names == {"linear", "linear_dz", "gated", "gated_dg_du", "ffn_grads", "column_sum",
                     "grad_norm", "grad_scale", "pack"}
    assert lib.lce_kernel_name(20) is None


@pytest.mark.parametrize("dt,mult", [(0, 8), (1, 4)])
def test_width_rule_is_sixteen_bytes_a_row(lib, dt, mult):
    for w in range(1, 33):
        ok = w % mult == 0
        assert (lib.lce_linear_workspace_size(10, w, 64, 0, 0, dt) > 0) == ok
        assert (lib.lce_linear_workspace_size(10, 64, w, 3, 1, dt) > 0) == ok
        assert (lib.lce_gated_workspace_size(10, w, 64, 0, dt) > 0) == ok
        assert (lib.lce_gated_workspace_size(10, 64, w, 1, dt) > 0) == ok


def test_workspace_size_refusals(lib):
    assert lib.lce_linear_workspace_size(-1, 64, 64, 0, 0, 0) == 0
    assert lib.lce_linear_workspace_size(1 << 31, 64, 64, 0, 0, 0) == 0
    assert lib.lce_linear_workspace_size(4, 0, 64, 0, 0, 0) == 0
    assert lib.lce_linear_workspace_size(4, 64, 1 << 31, 0, 0, 0) == 0
    assert lib.lce_linear_workspace_size((1 << 31) - 511, 64, 64, 0, 0, 0) == 0
    assert lib.lce_linear_workspace_size(1 << 30, 1 << 30, 64, 0, 0, 1) == 0     # 2^60 elements
    assert lib.lce_gated_workspace_size(64, 1 << 30, 1 << 30, 1, 0) == 0
    assert lib.lce_linear_workspace_size(4, 64, 64, 5, 0, 0) == 0      # activation
    assert lib.lce_linear_workspace_size(4, 64, 64, -1, 0, 0) == 0
    assert lib.lce_linear_workspace_size(4, 64, 64, 0, 2, 0) == 0      # direction
    assert lib.lce_linear_workspace_size(4, 64, 64, 0, 0, 2) == 0      # tf32x3 is not a type here
    assert lib.lce_gated_workspace_size(4, 64, 64, 0, 2) == 0
    assert lib.lce_gated_workspace_size(0, 64, 64, 1, 0) > 0           # no token is allowed
    assert lib.lce_grad_norm_workspace_size(-1) == 0
    assert lib.lce_grad_norm_workspace_size(0) > 0


def test_workspace_sizes(lib):
    """What the workspace holds: the header; the pre-activations' gradients in rows of whole 128-byte
    lines; for fp32 three bf16 parts of the operands; aligned copies where rows are no multiple of 32
    bytes and every element enters many products."""
    r64 = lambda x: (x + 63) // 64 * 64  # noqa: E731
    r256 = lambda x: (x + 255) // 256 * 256  # noqa: E731
    H = 256
    assert lib.lce_linear_workspace_size(5000, 4096, 4096, 3, 0, 0) == H
    assert lib.lce_linear_workspace_size(5000, 4096, 4096, 0, 1, 0) == H
    assert lib.lce_linear_workspace_size(5000, 4096, 4104, 3, 1, 0) == H + r256(5000 * r64(4104) * 2)
    assert lib.lce_gated_workspace_size(300, 64, 200, 1, 0) == H + 2 * r256(300 * r64(200) * 2)
    copies = r256(5000 * r64(4104) * 2) + r256(4096 * r64(4104) * 2)
    assert lib.lce_linear_workspace_size(5000, 4104, 4096, 3, 0, 0) == H + copies
    assert lib.lce_linear_workspace_size(50, 4104, 4096, 3, 0, 0) == H
    parts = lambda n, c: r256(n * r64(c) * 2 * 3)  # noqa: E731
    assert lib.lce_linear_workspace_size(8, 100, 200, 3, 0, 1) == H          # few tokens: no parts
    assert lib.lce_linear_workspace_size(80, 100, 200, 0, 0, 1) == H         # a small product: none either
    assert lib.lce_linear_workspace_size(800, 1000, 2000, 0, 0, 1) == H + parts(800, 1000) + parts(2000, 1000)
    assert lib.lce_gated_workspace_size(80, 100, 200, 1, 1) == \
        H + parts(80, 100) + 2 * parts(200, 100) + 2 * parts(80, 200)


def _linear(lib, X=P, ldx=64, W=P, b=P, R=P, ldr=96, N=5, di=64, do=96, act=0, dt=0, Y=P + 4096, ldy=96,
            ws=P, wsb=BIG):
    return lib.lce_linear_forward(X, ldx, W, b, R, ldr, N, di, do, act, dt, Y, ldy, ws, wsb, None)


def test_linear_forward_refusals(lib):
    assert _linear(lib, dt=2) == 1 and _linear(lib, dt=7) == 1 and _linear(lib, act=9) == 1
    assert _linear(lib, X=None) == 1 and _linear(lib, W=None) == 1 and _linear(lib, Y=None) == 1
    assert _linear(lib, ws=None) == 1
    for name in ("X", "W", "b", "R", "Y", "ws"):
        assert _linear(lib, **{name: P + 8}) == 1, name          # misaligned
    assert _linear(lib, di=60, ldx=64) == 2 and _linear(lib, do=95) == 2
    assert _linear(lib, ldx=56) == 2 and _linear(lib, ldx=68) == 2   # too short, not whole 16 bytes
    assert _linear(lib, ldy=88) == 2 and _linear(lib, ldr=88) == 2
    assert _linear(lib, N=-1) == 2
    assert _linear(lib, wsb=16) == 3
    assert _linear(lib, R=P + 4096, ldr=104) == 1                # in place with other row strides
    assert _linear(lib, Y=P) == 1                                # Y on top of X


def test_linear_backward_refusals(lib):
    def f(X=P, ldx=64, W=P, b=P, dY=P, ldy=96, N=5, act=2, dt=0, dX=P, dW=P, db=P, ws=P, wsb=BIG):
        return lib.lce_linear_backward(X, ldx, W, b, dY, ldy, N, 64, 96, act, dt, dX, dW, db, ws,
                                       wsb, None)
    assert f(act=-1) == 1 and f(dt=3) == 1
    for name in ("X", "W", "dY", "ws"):
        assert f(**{name: None}) == 1, name
    for name in ("X", "W", "b", "dY", "dX", "dW", "db", "ws"):
        assert f(**{name: P + 2}) == 1, name
    assert f(ldx=32) == 2 and f(ldy=95) == 2
    assert f(wsb=256) == 3                                        # the pre-activations' gradient


def test_gated_refusals(lib):
    def f(X=P, ldx=64, Wg=P, Wu=P, N=5, d=64, F=96, act=2, dt=0, H=P + 4096, ldh=96, ws=P, wsb=BIG):
        return lib.lce_gated_forward(X, ldx, Wg, Wu, N, d, F, act, dt, H, ldh, ws, wsb, None)

    def b(X=P, ldx=64, Wg=P, Wu=P, dH=P, ldh=96, dX=P, dWg=P, dWu=P, ws=P, wsb=BIG, act=2, dt=0):
        return lib.lce_gated_backward(X, ldx, Wg, Wu, dH, ldh, 5, 64, 96, act, dt, dX, dWg, dWu, ws,
                                      wsb, None)
    assert f(act=6) == 1 and f(dt=2) == 1
    for name in ("X", "Wg", "Wu", "H", "ws"):
        assert f(**{name: None}) == 1 and f(**{name: P + 4}) == 1, name
    assert f(d=62) == 2 and f(F=100) == 2 and f(ldx=60) == 2 and f(ldh=64) == 2 and f(wsb=0) == 3
    for name in ("X", "Wg", "Wu", "dH", "ws"):
        assert b(**{name: None}) == 1 and b(**{name: P + 4}) == 1, name
    assert b(dWg=None) == 1 and b(dWu=None) == 1                  # one weight gradient alone
    assert b(wsb=300) == 3 and b(ldh=40) == 2


def test_clip_refusals(lib):
    def f(ptrs=(P,), numels=(4,), dts=(1,), count=None, norm=0, m=1.0, total=P, ws=P, wsb=BIG, out=None):
        n = len(ptrs)
        o = None if out is None else (ctypes.c_void_p * n)(*out)
        return lib.lce_clip_grad_norm((ctypes.c_void_p * n)(*ptrs), o, (ctypes.c_int64 * n)(*numels),
                                      (ctypes.c_int32 * n)(*dts), n if count is None else count, norm, m,
                                      total, ws, wsb, None)
    assert f(norm=2) == 1 and f(m=-1.0) == 1 and f(m=float("nan")) == 1
    assert f(count=-1) == 1 and f(total=None) == 1 and f(ws=None) == 1 and f(ws=P + 4) == 1
    assert f(dts=(2,)) == 1                                       # type
    assert f(ptrs=(None,)) == 1 and f(ptrs=(P + 2,)) == 1         # null, misaligned fp32
    assert f(out=(None,)) == 1
    assert f(numels=(-1,)) == 2
    assert f(wsb=8) == 3


def test_python_refusals():
    x, w = torch.zeros(4, 64), torch.zeros(96, 64)
    with pytest.raises(ValueError, match="CUDA"):
        api.lce_linear_forward(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        api.lce_gated_forward(x, w, w)
    with pytest.raises(ValueError, match="CUDA"):
        api.lce_grad_norm([x])
    with pytest.raises(ValueError, match="no gradients"):
        api.lce_clip_grad_norm([], 1.0)
    with pytest.raises(ValueError, match="max_norm"):
        api.lce_clip_grad_norm([x], float("nan"))
    with pytest.raises(ValueError, match="norm must be"):
        api.lce_grad_norm([x], norm="l1")
    with pytest.raises(ValueError, match="x \\[..., d\\]"):
        api.linear_act(x, torch.zeros(96, 32))
    with pytest.raises(ValueError, match="residual"):
        api.linear_act(x, w, residual=torch.zeros(4, 1))
    p = torch.nn.Parameter(torch.zeros(3))
    assert api.clip_grad_norm_([p], 1.0).item() == 0.0            # no gradient anywhere
