"""Inputs and comparisons shared by the GPU tests of the gated recurrence and
the block norms."""
from __future__ import annotations

import numpy as np

import block_ref as ref

TYPES = {"f32": "float32", "bf16": "bfloat16", "f16": "float16"}


def torch_type(dtype):
    import torch
    return getattr(torch, TYPES[dtype])


def put(a, dtype="f32"):
    """A GPU tensor of the values, rounded to the type."""
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(torch_type(dtype)).cuda()


def back(t):
    import torch
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def column_slice(t, extra=3, offset=1):
    """The same values as a column range of a wider buffer of NaN: rows strided, and the
    first element off every wider alignment."""
    import torch
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, offset:offset + t.shape[1]] = t
    return wide[:, offset:offset + t.shape[1]], wide


def outside_is_nan(wide, width, offset=1):
    import torch
    return bool(torch.isnan(wide[:, :offset]).all() and torch.isnan(wide[:, offset + width:]).all())


def check(got, want, bound, dtype, what):
    """|got - want| within the fp32 bound plus one rounding to the output's type."""
    got = back(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    if want.size == 0:
        return 0.0
    tol = ref.tolerance(want, bound, dtype)
    err = np.abs(got - want)
    bad = ~(err <= tol)
    worst = float((err / tol)[~bad].max()) if (~bad).any() else 0.0
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first at "
                           f"{tuple(np.argwhere(bad)[0])}: got {got[bad][0]!r}, want {want[bad][0]!r}, "
                           f"tolerance {tol[bad][0]:.3g}")
    return worst


def gated_inputs(rng, B, L, D, gate, z=True, h0=True, reset=False, decay_mean=-3.0):
    n = lambda *s, m=0.0, sd=1.0: rng.normal(m, sd, size=s)
    M = B * L
    a = dict(x=n(M, D), r=n(M, D, m=1.0), i=None, decay=None, z=None, h0=None, reset=None)
    if gate == "log":
        a["r"] = -np.exp(n(M, D, m=-2.0))
    if gate == "decay":
        a["i"], a["decay"] = n(M, D), n(D, m=decay_mean)
    if z:
        a["z"] = n(M, D)
    if h0:
        a["h0"] = n(B, D)
    if reset:
        a["reset"] = (rng.random(M) < 0.05).astype(np.uint8)
    return a


ACTIVATIONS = ("x", "r", "i", "z", "dout")


def to_gpu(a, dtype):
    """GPU tensors of the inputs, and the inputs as the GPU holds them in fp64."""
    import torch
    g = {}
    for k, v in a.items():
        if k == "reset":
            g[k] = None if v is None else torch.from_numpy(v).cuda()
        else:
            g[k] = put(v, dtype if k in ACTIVATIONS else "f32")
    exact = {k: (a[k] if k == "reset" else back(v)) for k, v in g.items()}
    return g, exact
