"""NaN and infinities in the gated recurrence's inputs: outputs and gradients
are non-finite exactly where the definition makes them so, wherever the
kernels cut time, and right elsewhere."""
from __future__ import annotations

import numpy as np
import pytest

import block_ref as ref
import mamba_selective_scan_causal_amd as mss
from block_util import back, gated_inputs, to_gpu
from gpu_util import announce

pytestmark = pytest.mark.gpu

GATES = ("sigmoid", "decay", "log")
ROWS = ("y", "dx", "dr", "di", "dz")


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


def finite_where_defined(got, want, bound, dtype, what):
    got, ok = back(got), np.isfinite(want)
    extra, missing = ok & ~np.isfinite(got), ~ok & np.isfinite(got)
    assert not extra.any(), f"{what}: {extra.sum()} non-finite values, first at {tuple(np.argwhere(extra)[0])}"
    assert not missing.any(), f"{what}: {missing.sum()} finite values, first at {tuple(np.argwhere(missing)[0])}"
    with np.errstate(invalid="ignore", over="ignore"):
        bad = ok & ~(np.abs(got - want) <= ref.tolerance(want, bound, dtype))
    assert not bad.any(), (f"{what}: {bad.sum()} outside, first at {tuple(np.argwhere(bad)[0])}: got "
                           f"{got[bad][0]!r}, want {want[bad][0]!r}")


def far_gates(val, tol):
    """The bounds of a LOG gate with r below -40, which the reference's do not cover.

    log2(e) r is off by at most 1.5 |r| U of itself (the product's rounding, U, and the constant's,
    below U / 2), so a = 2^(log2(e) r) by 1.5 |r| U and an ulp, 2 U: for r >= -87.4 that is 133 U,
    within 3 K U = 192 U.  Below, a < 2^-126 is 0 in fp32: with G = dx and the state h that loses at
    most 2^-126 |G h| of dr, 2^-126 |h| of y (no z) and 2^-126 |G| of what the adjoint hands on."""
    most = {k: float(np.abs(val[k][np.isfinite(val[k])]).max()) for k in ("dx", "h")}
    lost = 2.0 ** -126 * (1 + most["dx"]) * (1 + most["h"])
    for k in tol:
        tol[k] = 3 * tol[k] + lost


def run(a, B, L, gate, dtype):
    """Every output and gradient against the fp64 form."""
    import torch
    g, e = to_gpu(a, dtype)
    kw = dict(batch=B, seq_len=L, gate=gate)
    y, ck, hl = mss.gated_scan(g["x"], g["r"], g["i"], g["decay"], g["z"], g["h0"], g["reset"], h_ckpt=True,
                               h_last=True, **kw)
    got = mss.gated_scan_backward(g["x"], g["r"], g["i"], g["decay"], g["z"], g["reset"], ck, g["dout"],
                                  dh_last=g["dh_last"], need_dh0=True, **kw)
    torch.cuda.synchronize()
    got.update(y=y, h_last=hl)
    with np.errstate(all="ignore"):
        val, tol = ref.gated_scan(**e, **kw)
    if gate == "log":
        far_gates(val, tol)
    for k, v in got.items():
        if v is not None:
            finite_where_defined(v, val[k], tol[k], dtype if k in ROWS else "f32", k)


def inputs(seed, B, L, D, gate, **opt):
    rng = np.random.default_rng(seed)
    # gates around 1/2: the product over some hundred steps is 0 in fp32
    a = gated_inputs(rng, B, L, D, gate, decay_mean=-1.0, **opt)
    a["r"] = -np.exp(rng.normal(size=(B * L, D))) if gate == "log" else rng.normal(size=(B * L, D))
    a["dout"], a["dh_last"] = rng.normal(size=(B * L, D)), rng.normal(size=(B, D))
    return a


# 2 and 13 tiles of channels: the two sizes of the groups that chunks are
# handed over in
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("D", (70, 832))
@pytest.mark.parametrize("bad", (np.nan, np.inf, -np.inf))
def test_what_the_state_carries_stays_to_the_end(gate, D, bad):
    """One bad input in each of a few channels, and no reset behind it."""
    L = 5120
    a = inputs(3, 1, L, D, gate, z=False, h0=True)
    a["x"][300, 5], a["x"][4000, 6], a["x"][127, 7], a["x"][128, 8], a["h0"][0, 9] = (bad,) * 5
    run(a, 1, L, gate, "f32")


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("D", (70, 832))
@pytest.mark.parametrize("bad", (np.nan, np.inf, -np.inf))
def test_what_the_adjoint_carries_stays_to_the_start(gate, D, bad):
    L = 2560
    a = inputs(4, 1, L, D, gate, z=False, h0=True)
    a["dout"][2300, 5], a["dout"][64, 6], a["dout"][63, 7], a["dout"][1000, 8], a["dh_last"][0, 9] = (bad,) * 5
    run(a, 1, L, gate, "f32")


@pytest.mark.parametrize("gate", GATES)
def test_bad_values_end_at_a_reset(gate):
    """The same with resets: the states before and after are those without the bad values."""
    L, D = 2560, 70
    a = inputs(5, 1, L, D, gate, z=False, h0=True, reset=False)
    a["x"][300, 5], a["x"][700, 6], a["dout"][2300, 7], a["dout"][1200, 5] = np.nan, np.inf, np.nan, np.inf
    a["reset"] = np.zeros(L, np.uint8)
    a["reset"][[290, 1000, 2200]] = 1
    with np.errstate(all="ignore"):
        run_with_resets(a, L, D, gate)


def run_with_resets(a, L, D, gate):
    """The reference multiplies by 0 where a state is dropped, which a NaN survives: each document
    is taken alone."""
    import torch
    g, e = to_gpu(a, "f32")
    kw = dict(batch=1, gate=gate)
    y, ck, hl = mss.gated_scan(g["x"], g["r"], g["i"], g["decay"], None, g["h0"], g["reset"], seq_len=L, h_ckpt=True,
                               h_last=True, **kw)
    got = mss.gated_scan_backward(g["x"], g["r"], g["i"], g["decay"], None, g["reset"], ck, g["dout"],
                                  dh_last=g["dh_last"], need_dh0=True, seq_len=L, **kw)
    torch.cuda.synchronize()
    starts = [0, *np.flatnonzero(e["reset"]), L]
    for s, t in zip(starts, starts[1:]):
        part = {k: None if e[k] is None else e[k][s:t] for k in ("x", "r", "i", "dout")}
        val, tol = ref.gated_scan(**part, decay=e["decay"], h0=e["h0"] if s == 0 else None, seq_len=t - s,
                                  dh_last=e["dh_last"] if t == L else None, **kw)
        if gate == "log":
            far_gates(val, tol)
        finite_where_defined(y[s:t], val["y"], tol["y"], "f32", f"y from {s}")
        for k in ("dx", "dr", "di"):
            if got[k] is not None:
                finite_where_defined(got[k][s:t], val[k], tol[k], "f32", f"{k} from {s}")
        if s == 0:
            finite_where_defined(got["dh0"], val["dh0"], tol["dh0"], "f32", "dh0")
    finite_where_defined(hl, val["h_last"], tol["h_last"], "f32", "h_last")


@pytest.mark.parametrize("gate,which", [("decay", "r"), ("decay", "i"), ("sigmoid", "r"), ("log", "r"),
                                        ("decay", "decay"), ("sigmoid", "z")])
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("L", (60, 300))
def test_a_nan_gate_reaches_the_gradients(gate, which, dtype, L):
    """A gate that is NaN in one step of a few channels makes that step's gradients NaN, and with them
    what the recurrence makes of it before and after."""
    B, D = 2, 33
    a = inputs(6, B, L, D, gate, z=which in ("i", "z"), h0=True)
    if which == "decay":
        a["decay"][[3, 8]] = np.nan
    else:
        a[which][[20, 41], [5, 6]] = np.nan
        a[which][L + 17, 5] = np.nan
    run(a, B, L, gate, dtype)
