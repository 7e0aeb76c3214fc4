"""What is measured of the feed-forward operators and of gradient clipping.

Three operators, each in the directions a training run and a server use it:

* ``gated``   H = act(X Wg^T) * (X Wu^T), the gated feed-forward's first half; its backward pass
              (dX, dWg, dWu from X, Wg, Wu and dH); its form for a few tokens.
* ``linear``  Y = act(X W^T + b) + R, the product with bias, activation and residual in its
              epilogue; its backward pass (dX, dW, db; the gradient of R is dY itself); its form
              for a few tokens.
* ``clip``    the global 2-norm over many gradient tensors and their scaling to a largest norm.

A case is a dict of plain values; ``kind`` names the operator and ``way`` its direction ("fwd" or
"bwd").  Sizes are in elements: N tokens, d the model width, F the feed-forward width (for
``linear``: d_in -> d_out).
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
# The largest pass of each kind, in multiply-adds of one product over N x d x F (clip: elements).
LARGEST = {"gated": 16384 * 4096 * 16384, "linear": 16384 * 4096 * 16384, "clip": 320_000_000}
# float32 products cost several tensor-core products each: their range ends earlier.
LARGEST_F32 = 2048 * 2048 * 8192


def listed():
    return [
        # one token being decoded, the width of the N=4096 workload and four times it
        dict(name="gated-decode-1", kind="gated", way="fwd", dtype="bf16", act="silu", N=1, d=2048, F=8192),
        # a batch of sequences being decoded together, the widest model of the workloads
        dict(name="gated-decode-48", kind="gated", way="fwd", dtype="bf16", act="silu", N=48, d=6144, F=16384),
        # a prompt of odd length and a feed-forward width that ends inside a tile
        dict(name="gated-prompt-777", kind="gated", way="fwd", dtype="bf16", act="gelu_tanh", N=777, d=4096, F=10952),
        # the backward pass of a training step at the tokens and width of the N=16384 workload
        dict(name="gated-train-16384", kind="gated", way="bwd", dtype="bf16", act="silu", N=16384, d=4096, F=16384),
        # a small float32 model, odd sizes
        dict(name="gated-train-f32", kind="gated", way="bwd", dtype="f32", act="gelu", N=601, d=260, F=1004),
        # the second half of the block for four tokens: no activation, added to the residual
        dict(name="linear-decode-4", kind="linear", way="fwd", dtype="bf16", act="none", bias=False, residual=True,
             N=4, d_in=16384, d_out=4096),
        # the second half of the block in a training step's forward pass
        dict(name="linear-down-4096", kind="linear", way="fwd", dtype="bf16", act="none", bias=True, residual=True,
             N=4096, d_in=8192, d_out=2048),
        # a dense transform in float32 for two tokens
        dict(name="linear-decode-f32", kind="linear", way="fwd", dtype="f32", act="gelu", bias=True, residual=False,
             N=2, d_in=2048, d_out=2048),
        # the backward pass of a dense transform with activation, an odd number of tokens
        dict(name="linear-train-4095", kind="linear", way="bwd", dtype="bf16", act="gelu", bias=True, residual=False,
             N=4095, d_in=2048, d_out=8192),
        # a small float32 model's gradients, where latency counts: 27 tensors, some of one element
        dict(name="clip-small", kind="clip", way="fwd", tensors=27, total=300_000, wide=0),
        # the gradients of a few feed-forward blocks in bfloat16 with float32 vectors between them
        dict(name="clip-blocks", kind="clip", way="fwd", tensors=20, total=100_000_000, wide=0),
        # those next to a vocabulary projection's float32 gradient (151936 x 2048)
        dict(name="clip-vocabulary", kind="clip", way="fwd", tensors=9, total=8_000_000, wide=311_164_928),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(n, step):
    """n rounded to a multiple of step."""
    n = max(step, n // step * step)
    return n + step if n == 3072 else n


def draw(rng):
    kind = rng.choice(["gated", "gated", "linear", "linear", "clip"])
    if kind == "clip":
        total = _log(rng, 1_000, 150_000_000)
        wide = _log(rng, 1_000_000, 150_000_000) if rng.random() < 0.4 else 0
        return dict(kind=kind, way="fwd", tensors=rng.randint(2, 40), total=total, wide=wide)
    way = rng.choice(["fwd", "fwd", "bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    step = 8 if dtype == "bf16" else 4
    most = LARGEST[kind] if dtype == "bf16" else LARGEST_F32
    if way == "fwd" and rng.random() < 0.5:
        N = _log(rng, 1, 128)
    else:
        N = _size(_log(rng, 65, 16384), 1)
    a, b = _size(_log(rng, 256, 6144), step), _size(_log(rng, 512, 16384), step)
    while N * a * b > most:
        N = max(1, N * 3 // 4)
        b = _size(b * 7 // 8, step)
    N = _size(N, 1)
    if kind == "gated":
        return dict(kind=kind, way=way, dtype=dtype, act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"]), N=N, d=a, F=b)
    if rng.random() < 0.5:
        a, b = b, a
    return dict(kind=kind, way=way, dtype=dtype, act=rng.choice(["none", "none", "gelu", "silu", "relu"]),
                bias=rng.random() < 0.5, residual=way == "fwd" and rng.random() < 0.5, N=N, d_in=a, d_out=b)


# ------------------------------------------------------------------------------------ inputs

def _numels(case):
    """Sizes and types of a clip case's tensors: vectors of a few elements in float32 between
    matrices whose sizes spread by a factor of 30, in bfloat16."""
    r = np.random.RandomState(case["tensors"] * 7919 + case["total"] % 65521)
    share = np.exp(r.uniform(0.0, math.log(30.0), case["tensors"]))
    out = []
    for k in range(case["tensors"]):
        if k % 3 == 1:
            out.append((int(r.randint(1, 4097)), torch.float32))
        else:
            out.append((max(1, int(case["total"] * share[k] / share.sum())), torch.bfloat16))
    if case["wide"]:
        out.append((int(case["wide"]), torch.float32))
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype):
        t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
        return t.mul_(std).to(dtype)

    st = dict(case=dict(case))
    if case["kind"] == "clip":
        numels = _numels(case)
        n = sum(k for k, _ in numels)
        # a norm of about 3.3: clipped to 1, as in the noisy steps where clipping acts
        st["grads"] = [normal(k, std=3.3 / math.sqrt(n), dtype=dt) for k, dt in numels]
        st["clipped"] = [torch.empty_like(t) for t in st["grads"]]
        return st
    dt = DTYPES[case["dtype"]]
    N = case["N"]
    d_in, d_out = (case["d"], case["F"]) if case["kind"] == "gated" else (case["d_in"], case["d_out"])
    x = torch.randn(N, d_in, generator=g, device="cuda", dtype=torch.float32)
    # a few features far above the rest, as hidden states have
    x[:, torch.randperm(d_in, generator=g, device="cuda")[:max(1, d_in // 256)]] *= 6.0
    st["x"] = x.to(dt)
    del x
    w = 1.0 / math.sqrt(d_in)
    st["w"] = normal(d_out, d_in, std=w, dtype=dt)
    if case["kind"] == "gated":
        st["wu"] = normal(d_out, d_in, std=w, dtype=dt)
    st["bias"] = normal(d_out, std=0.1, dtype=dt) if case.get("bias") else None
    st["residual"] = normal(N, d_out, dtype=dt) if case.get("residual") else None
    if case["way"] == "bwd":
        st["dy"] = normal(N, d_out, std=1.0 / N, dtype=dt)
    return st


# ------------------------------------------------------------------------------------ passes

def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    from memory_bounded_linear_gb300 import api
    case = st["case"]
    if case["kind"] == "clip":
        total, clipped, _ = api.lce_clip_grad_norm(st["grads"], 1.0, out=st["clipped"])
        return {"total": total, "clipped": clipped}
    if case["kind"] == "gated":
        if case["way"] == "fwd":
            return api.lce_gated_forward(st["x"], st["w"], st["wu"], activation=case["act"])[0]
        dx, dwg, dwu, _ = api.lce_gated_backward(st["x"], st["w"], st["wu"], st["dy"], activation=case["act"])
        return {"dx": dx, "dwg": dwg, "dwu": dwu}
    if case["way"] == "fwd":
        return api.lce_linear_forward(st["x"], st["w"], st["bias"], st["residual"], activation=case["act"])[0]
    dx, dw, db, _ = api.lce_linear_backward(st["x"], st["w"], st["bias"], st["dy"], activation=case["act"])
    return {"dx": dx, "dw": dw, "db": db}


def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z * (1.0 / (1.0 + torch.exp(-z)))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    u = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)
    return 0.5 * z * (1.0 + torch.tanh(u))


def _act_grad(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)


def _plain(st):
    case = st["case"]
    if case["kind"] == "clip":
        total = torch.stack([t.float().square().sum() for t in st["grads"]]).sum().sqrt()
        coef = torch.clamp(1.0 / (total + 1e-6), max=1.0)
        return {"total": total, "clipped": [(t.float() * coef).to(t.dtype) for t in st["grads"]]}
    dt = st["x"].dtype
    x, w = st["x"].float(), st["w"].float()
    if case["kind"] == "gated":
        wu = st["wu"].float()
        g, u = x @ w.t(), x @ wu.t()
        if case["way"] == "fwd":
            return (_act(g, case["act"]) * u).to(dt)
        dy = st["dy"].float()
        dg = dy * u * _act_grad(g, case["act"])
        du = dy * _act(g, case["act"])
        dx = (dg @ w + du @ wu).to(dt)
        return {"dx": dx, "dwg": (dg.t() @ x).to(dt), "dwu": (du.t() @ x).to(dt)}
    z = None
    if case["way"] == "fwd" or case["act"] != "none":
        z = x @ w.t()
        if st["bias"] is not None:
            z = z + st["bias"].float()
    if case["way"] == "fwd":
        y = _act(z, case["act"])
        if st["residual"] is not None:
            y = y + st["residual"].float()
        return y.to(dt)
    dy = st["dy"].float()
    dz = dy if z is None else dy * _act_grad(z, case["act"])
    return {"dx": (dz @ w).to(dt), "dw": (dz.t() @ x).to(dt),
            "db": dz.sum(0).to(dt) if st["bias"] is not None else None}


# ------------------------------------------------------------------------------------ the work

def work(case):
    """Bytes: every input read once, every output written once.  Operations: the products (the
    backward pass is given X, the weights and the outgoing gradient, so the pre-activations that
    the activation's gradient needs are a product of their own) and a few per element."""
    if case["kind"] == "clip":
        numels = _numels(case)
        size = sum(n * (2 if dt == torch.bfloat16 else 4) for n, dt in numels)
        return {"bytes": 2 * size + 4, "flops": 3 * sum(n for n, _ in numels)}
    e = 2 if case["dtype"] == "bf16" else 4
    N = case["N"]
    if case["kind"] == "gated":
        d, F = case["d"], case["F"]
        weights, x, h = 2 * d * F, N * d, N * F
        if case["way"] == "fwd":
            return {"bytes": e * (weights + x + h), "flops": 4 * N * d * F}
        return {"bytes": e * (2 * weights + 2 * x + h), "flops": 12 * N * d * F}
    a, b = case["d_in"], case["d_out"]
    bias = b if case["bias"] else 0
    if case["way"] == "fwd":
        return {"bytes": e * (a * b + N * a + N * b * (2 if case["residual"] else 1) + bias), "flops": 2 * N * a * b}
    inputs = a * b + N * a + N * b + (bias if case["act"] != "none" else 0)
    return {"bytes": e * (inputs + a * b + N * a + bias), "flops": (4 if case["act"] == "none" else 6) * N * a * b}


# ------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    st = prepare(case, seed)
    if case["kind"] == "clip":
        squares = 0.0
        for t in st["grads"]:
            for part in t.split(1 << 26):
                squares += float((part.double() ** 2).sum())
        total = math.sqrt(squares)
        coef = min(1.0, 1.0 / (total + 1e-6))
        return {"total": torch.tensor(total, dtype=torch.float64), "clipped": [t.double() * coef for t in st["grads"]]}
    x, w = st["x"].double(), st["w"].double()
    z = torch.einsum("nk,mk->nm", x, w)
    if st["bias"] is not None:
        z += st["bias"].double()
    zv = z.detach().requires_grad_(True)
    act = case["act"]
    if act == "none":
        a = zv * 1.0
    elif act == "relu":
        a = torch.clamp(zv, min=0.0)
    elif act == "silu":
        a = zv / (1.0 + torch.exp(-zv))
    elif act == "gelu":
        a = zv * 0.5 * torch.erfc(-zv / math.sqrt(2.0))
    else:
        # 0.5 (1 + tanh(u)) = 1 / (1 + exp(-2u))
        a = zv / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (zv + 0.044715 * zv ** 3)))
    if case["kind"] == "gated":
        wu = st["wu"].double()
        u = torch.einsum("nk,mk->nm", x, wu)
        if case["way"] == "fwd":
            return a.detach() * u
        dy = st["dy"].double()
        dg = torch.autograd.grad(a, zv, dy * u)[0]
        du = dy * a.detach()
        dx = torch.einsum("nm,mk->nk", dg, w) + torch.einsum("nm,mk->nk", du, wu)
        return {"dx": dx, "dwg": torch.einsum("nm,nk->mk", dg, x), "dwu": torch.einsum("nm,nk->mk", du, x)}
    if case["way"] == "fwd":
        y = a.detach()
        return y + st["residual"].double() if st["residual"] is not None else y
    dz = torch.autograd.grad(a, zv, st["dy"].double())[0]
    return {"dx": torch.einsum("nm,mk->nk", dz, w), "dw": torch.einsum("nm,nk->mk", dz, x),
            "db": dz.sum(0) if st["bias"] is not None else None}
