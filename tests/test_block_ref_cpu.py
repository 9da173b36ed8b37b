"""The fp64 forms that the GPU tests of the gated recurrence and the block
norms compare with, checked on the CPU: closed forms, and every gradient
against central differences."""
from __future__ import annotations

import numpy as np
import pytest

import block_ref as ref


def close(got, want, tol=1e-7):
    assert np.abs(got - want).max() <= tol * max(1.0, np.abs(want).max())


def test_closed_forms():
    L, D = 7, 3
    x = np.ones((L, D))
    # constant a: a geometric series
    a = 0.25
    val, _ = ref.gated_scan(x, np.full((L, D), np.log(a)), batch=1, seq_len=L, gate="log")
    close(val["h"][0, :, 0], (1 - a ** np.arange(1, L + 1)) / (1 - a), 1e-14)
    # sigmoid gates average: constant x stays, h0 = x
    val, _ = ref.gated_scan(3 * x, np.random.default_rng(0).normal(size=(L, D)), h0=np.full((1, D), 3.0),
                            batch=1, seq_len=L, gate="sigmoid")
    close(val["y"], 3 * x, 1e-14)
    # r = -inf: nothing is carried; for the decay gate nothing is let in
    inf = np.full((L, D), -np.inf)
    for gate in ("sigmoid", "log"):
        close(ref.gated_scan(x, inf, h0=x[:1], batch=1, seq_len=L, gate=gate)[0]["h_last"], x[:1])
    got = ref.gated_scan(x, inf, x, np.zeros(D), h0=x[:1] * 5, batch=1, seq_len=L, gate="decay")[0]
    close(got["h_last"], 5 * x[:1])
    # a reset equals two sequences
    rng = np.random.default_rng(1)
    x, r = rng.normal(size=(2, L, D))
    reset = np.zeros(L, np.uint8)
    reset[3] = 1
    whole = ref.gated_scan(x, r, reset=reset, batch=1, seq_len=L, gate="sigmoid")[0]
    tail = ref.gated_scan(x[3:], r[3:], batch=1, seq_len=L - 3, gate="sigmoid")[0]
    close(whole["y"][3:], tail["y"], 1e-15)


def differences(f, args, dargs):
    """Central differences of sum(f * cotangents) against the gradients given."""
    rng = np.random.default_rng(9)
    for name, grad in dargs.items():
        a = args[name]
        for _ in range(6):
            at = tuple(rng.integers(n) for n in a.shape)
            keep, e = a[at], 1e-5
            a[at] = keep + e
            up = f()
            a[at] = keep - e
            down = f()
            a[at] = keep
            close(np.array([grad[at]]), np.array([(up - down) / (2 * e)]), 2e-8)


@pytest.mark.parametrize("gate", ("sigmoid", "decay", "log"))
@pytest.mark.parametrize("gated", (False, True))
def test_scan_gradients_by_differences(gate, gated):
    rng = np.random.default_rng(3)
    B, L, D = 2, 6, 3
    a = dict(x=rng.normal(size=(B * L, D)), r=rng.normal(size=(B * L, D)), h0=rng.normal(size=(B, D)))
    if gate == "log":
        a["r"] -= 1.0
    if gate == "decay":
        a.update(i=rng.normal(size=(B * L, D)), decay=rng.normal(size=D) - 2)
    if gated:
        a["z"] = rng.normal(size=(B * L, D))
    dout, dhl = rng.normal(size=(B * L, D)), rng.normal(size=(B, D))
    reset = (rng.random(B * L) < 0.25).astype(np.uint8)
    kw = dict(reset=reset, batch=B, seq_len=L, gate=gate, gate_scale=3.0)

    def f():
        val, _ = ref.gated_scan(**a, **kw)
        return (val["y"] * dout).sum() + (val["h_last"] * dhl).sum()

    val, tol = ref.gated_scan(**a, dout=dout, dh_last=dhl, **kw)
    grads = {n: val["d" + n] for n in a}
    differences(f, a, grads)
    for n in val:
        assert (tol[n] <= 1e-3 * (1 + np.abs(val[n]).max())).all()


@pytest.mark.parametrize("kind", ("rms", "layer"))
def test_add_norm_gradients_by_differences(kind):
    rng = np.random.default_rng(4)
    M, D = 3, 5
    a = dict(x=rng.normal(size=(M, D)), residual=rng.normal(size=(M, D)), scale=rng.normal(size=D),
             weight=rng.normal(size=D), bias=rng.normal(size=D))
    dy, ds = rng.normal(size=(2, M, D))

    def f():
        s, _ = ref.add_norm(a["x"], a["residual"], a["scale"], 0.6)
        y, _ = ref.norm_of(s, a["weight"], a["bias"], kind, 1e-3)
        return (y * dy).sum() + (s * ds).sum()

    s, _ = ref.add_norm(a["x"], a["residual"], a["scale"], 0.6)
    val, _ = ref.add_norm_backward(s, a["weight"], dy, ds, a["x"], a["scale"], kind=kind, eps=1e-3,
                                   alpha=0.6)
    differences(f, a, {n: val["d" + n] for n in a})


@pytest.mark.parametrize("kind", ("rms", "layer"))
@pytest.mark.parametrize("order", ("before", "after"))
@pytest.mark.parametrize("gated", (False, True))
def test_gated_norm_gradients_by_differences(kind, order, gated):
    rng = np.random.default_rng(5)
    M, D = 3, 6
    a = dict(x=rng.normal(size=(M, D)), weight=rng.normal(size=D), bias=rng.normal(size=D),
             scale=rng.normal(size=D))
    if gated:
        a["z"] = rng.normal(size=(M, D))
    dout, residual = rng.normal(size=(2, M, D))
    kw = dict(groups=2, order=order, kind=kind, eps=1e-3, alpha=0.6)
    args = lambda: (a["x"], a.get("z"), a["weight"], a["bias"], residual, a["scale"])
    f = lambda: (ref.gated_norm(*args(), **kw)[0]["y"] * dout).sum()
    val, _ = ref.gated_norm(*args(), dout, **kw)
    differences(f, a, {n: val["d" + n] for n in a})
