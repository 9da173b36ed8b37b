"""Gates at the ends of their range: every output and every gradient of the
gated recurrence against the fp64 form, whose decay gate takes its limit where
its input scale vanishes."""
from __future__ import annotations

import numpy as np
import pytest

import block_ref as ref
import mamba_selective_scan_causal_amd as mss
from block_util import check, gated_inputs, to_gpu
from gpu_util import announce

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


def widen(e, val, tol, B, L, z):
    """What the reference's bounds of the decay gate leave out at the ends of its range.

    With Lam = k sigma(r) = -ln a, c max(1, softplus(decay)) <= 32.2 here, and S = the sum over later
    steps of the absolute terms of G:
      - the reference's UNDER, sqrt(64 2^-126), covers c softplus <= 32: sqrt(32.2 / 32) < 1.004 of it;
      - the backward holds sigma(r) and sigma(i) at 2^-126 or more: up to 2^-126 S of dx, 2^-126 S |x|
        of di, and of dr and ddecay 2^-126 times S k |h| <= 32.2 S |h| and S |x| Lam a^2 / m, where
        Lam a^2 / m = Lam e^(-2 Lam) / sqrt(1 - e^(-2 Lam)) <= 1 for every Lam >= 0;
      - where softplus(decay) or Lam is 0 in fp32 (below 2^-126), Lam a^2 / m <= sqrt(Lam / 2), which
        sums to c sigma(decay) q a^2 / m <= Lam a^2 / m in ddecay (sigma(d) <= softplus(d)), is lost:
        at most UNDER S |x| sigma(i) of it."""
    x, r, i = (np.asarray(e[k]).reshape(B, L, -1) for k in ("x", "r", "i"))
    a = np.exp(-8.0 * ref.softplus(e["decay"]) * ref.sigmoid(r))
    dy = np.abs(e["dout"].reshape(x.shape)) * (1.0 if z is None else np.abs(ref.silu(z.reshape(x.shape))))
    S, now = np.empty_like(x), np.abs(e["dh_last"])
    for t in range(L - 1, -1, -1):
        S[:, t] = dy[:, t] + now
        now = a[:, t] * S[:, t]
    small = 2.0 ** -126 * 33 * S * (1 + np.abs(x) + np.abs(val["h"]).max())
    for k in tol:
        tol[k] = 1.004 * tol[k]
    for k in ("dx", "dr", "di"):
        tol[k] = tol[k] + small.reshape(tol[k].shape)
    tol["ddecay"] = tol["ddecay"] + (small + ref.UNDER * S * np.abs(x) * ref.sigmoid(i)).sum((0, 1))


@pytest.mark.parametrize("gate,r,i", [
    ("sigmoid", (-np.inf, -200.0, 200.0, np.inf), ()), ("log", (-np.inf, -200.0), ()),
    ("decay", (-np.inf, -200.0, 200.0, np.inf), ()), ("decay", (), (-np.inf, -200.0, 200.0, np.inf)),
    ("decay", (-np.inf, -200.0, 200.0, np.inf), (-np.inf, -200.0, 200.0, np.inf))])
@pytest.mark.parametrize("dtype", ("f32", "bf16", "f16"))
@pytest.mark.parametrize("L,z", [(40, True), (330, False)])
def test_gates_at_their_ends(gate, r, i, dtype, L, z):
    import torch
    rng = np.random.default_rng(L)
    B, D = 2, 37
    a = gated_inputs(rng, B, L, D, gate, z=z, h0=True)
    for k, ends in (("r", r), ("i", i)):
        which = rng.integers(0, 8, size=(B * L, D))
        for n, v in enumerate(ends):
            a[k][which == n] = v
    if gate == "decay":
        a["decay"][::4], a["decay"][1::4], a["decay"][2::4] = -30.0, -120.0, 4.0
    a["dout"], a["dh_last"] = rng.normal(size=(B * L, D)), rng.normal(size=(B, D))
    g, e = to_gpu(a, dtype)
    kw = dict(batch=B, seq_len=L, gate=gate)
    y, ck, hl = mss.gated_scan(g["x"], g["r"], g["i"], g["decay"], g["z"], g["h0"], h_ckpt=True, h_last=True, **kw)
    got = mss.gated_scan_backward(g["x"], g["r"], g["i"], g["decay"], g["z"], None, ck, g["dout"],
                                  dh_last=g["dh_last"], need_dh0=True, **kw)
    torch.cuda.synchronize()
    val, tol = ref.gated_scan(**e, **kw)
    if gate == "decay":
        widen(e, val, tol, B, L, e["z"])
    check(y, val["y"], tol["y"], dtype, "y")
    check(hl, val["h_last"], tol["h_last"], "f32", "h_last")
    for k, v in got.items():
        if v is not None:
            check(v, val[k], tol[k], dtype if k in ("dx", "dr", "di", "dz") else "f32", k)
