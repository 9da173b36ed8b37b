"""The gated recurrence and the block norms at random sizes, types, strides and
options (fixed seeds), against the fp64 forms within their derived bounds."""
from __future__ import annotations

import numpy as np
import pytest

import block_ref as ref
import mamba_selective_scan_causal_amd as mss
from block_util import back, check, column_slice, gated_inputs, put, to_gpu, torch_type
from gpu_util import announce

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


def size(rng, low, high):
    return int(round(np.exp(rng.uniform(np.log(low), np.log(high)))))


def maybe_strided(rng, t):
    return t if t is None or rng.random() < 0.5 else column_slice(t, int(rng.integers(2, 9)), int(rng.integers(0, 3)))[0]


@pytest.mark.parametrize("seed", range(40))
def test_gated_scan(seed):
    import torch
    rng = np.random.default_rng(500 + seed)
    D, B = size(rng, 1, 700), int(rng.integers(1, 6))
    L = size(rng, 1, min(3000, 300000 // (B * D) + 1))
    gate, dtype = rng.choice(["sigmoid", "decay", "log"]), str(rng.choice(["f32", "bf16", "f16"]))
    opt = dict(z=rng.random() < 0.5, h0=rng.random() < 0.5, reset=rng.random() < 0.5)
    announce(f"B{B} L{L} D{D} {gate} {dtype} {opt}")
    a = gated_inputs(rng, B, L, D, gate, decay_mean=float(rng.uniform(-8, 0)), **opt)
    a["dout"] = rng.normal(size=(B * L, D))
    a["dh_last"] = rng.normal(size=(B, D)) if rng.random() < 0.5 else None
    g, e = to_gpu(a, dtype)
    scale = float(rng.uniform(0.5, 8))
    kw = dict(batch=B, seq_len=L, gate=str(gate), gate_scale=scale)
    s = {k: maybe_strided(rng, g[k]) if k in ("x", "r", "i", "z", "dout") else g[k] for k in g}
    y, ck, hl = mss.gated_scan(s["x"], s["r"], s["i"], s["decay"], s["z"], s["h0"], s["reset"], h_ckpt=True,
                               h_last=True, **kw)
    got = mss.gated_scan_backward(s["x"], s["r"], s["i"], s["decay"], s["z"], s["reset"], ck, s["dout"],
                                  dh_last=s["dh_last"], need_dh0=True, **kw)
    torch.cuda.synchronize()
    kw["gate_scale"] = float(np.float32(scale))
    val, tol = ref.gated_scan(**e, **kw)
    check(y, val["y"], tol["y"], dtype, "y")
    check(hl, val["h_last"], tol["h_last"], "f32", "h_last")
    for k, v in got.items():
        if v is not None:
            check(v, val[k], tol[k], dtype if k in ("dx", "dr", "di", "dz") else "f32", k)


@pytest.mark.parametrize("seed", range(40))
def test_norms(seed):
    import torch
    rng = np.random.default_rng(900 + seed)
    groups = int(rng.choice([1, 1, 2, 3, 8]))
    D = max(1, size(rng, 1, 13000) // groups) * groups
    M = size(rng, 1, min(2000, 400000 // D + 1))
    dtype, kind = str(rng.choice(["f32", "bf16", "f16"])), str(rng.choice(["rms", "layer"]))
    order = str(rng.choice(["before", "after"]))
    has = lambda: rng.random() < 0.5
    n = lambda *s: rng.normal(size=s)
    alpha = float(np.float32(rng.uniform(0.2, 1.5)))
    eps = float(np.float32(10.0 ** rng.uniform(-7, -3)))
    announce(f"M{M} D{D} groups {groups} {dtype} {kind} {order}")
    act = lambda t=dtype: maybe_strided(rng, put(n(M, D), t))
    x, z, res, dout = act(), act() if has() else None, act() if has() else None, act()
    w, b, sc = put(n(D)), put(n(D)) if has() else None, put(n(D)) if has() else None
    kw = dict(groups=groups, order=order, kind=kind, eps=eps, alpha=alpha)
    y = mss.gated_norm(x, z, w, b, res, sc, **kw)
    g = mss.gated_norm_backward(x, z, w, b, sc, dout, **kw)
    torch.cuda.synchronize()
    val, tol = ref.gated_norm(*(back(t) for t in (x, z, w, b, res, sc, dout)), **kw)
    check(y, val["y"], tol["y"], dtype, "y")
    for k, v in g.items():
        if v is not None:
            check(v, val[k], tol[k], dtype if k in ("dx", "dz") else "f32", k)
    rt = str(rng.choice(["f32", dtype]))
    old, up = act(rt) if has() else None, act(rt) if has() else None
    kw = dict(kind=kind, eps=eps, alpha=alpha)
    y, s = mss.add_norm(x, old, w, b, sc, res_dtype=torch_type(rt), **kw)
    g = mss.add_norm_backward(s, w, dout, up, x if sc is not None else None, sc, bias=b is not None, **kw)
    torch.cuda.synchronize()
    want, bound = ref.add_norm(back(x), back(old), back(sc), alpha)
    check(s, want, bound, rt, "s")
    want, bound = ref.norm_of(back(s), back(w), back(b), kind, eps)
    check(y, want, bound, dtype, "y")
    val, tol = ref.add_norm_backward(back(s), back(w), back(dout), back(up), back(x) if sc is not None else None,
                                     back(sc), **kw)
    for k, v in g.items():
        if v is not None:
            check(v, val[k], tol[k], dtype if k == "dx" else rt if k == "dresidual" else "f32", k)
