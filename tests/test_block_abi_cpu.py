"""Refusals of the gated recurrence and the block norms at the C ABI, without a
GPU: every call is rejected, or is empty, before any launch, so the pointers
are fake aligned addresses that are never dereferenced."""
from __future__ import annotations

import ctypes

import pytest

import mamba_selective_scan_causal_amd as mss

EINVAL, EALIGN, EALIAS, EWORKSPACE = -1, -2, -3, -4
BASE = 0x7F0000000000


def fake(i, off=0):
    return ctypes.c_void_p(BASE + i * (1 << 32) + off)


@pytest.fixture(scope="module")
def L():
    return mss.lib()


def gated(B=2, L=100, D=64, dtype=1, gate=1, scale=8.0):
    return mss.GatedDims(ctypes.sizeof(mss.GatedDims), 0, dtype, gate, B, L, D, scale, 0)


def norm(M=10, D=64, dtype=1, res=1, kind=0, order=0, groups=1, eps=1e-6, alpha=1.0):
    return mss.NormDims(ctypes.sizeof(mss.NormDims), 0, dtype, res, kind, order, M, D, groups, eps, alpha)


def strides(cls, value):
    s = cls()
    for name, _ in cls._fields_:
        setattr(s, name, value)
    s.struct_size, s.reserved = ctypes.sizeof(cls), 0
    return s


def need(L, dims, op):
    n = ctypes.c_size_t(7)
    f = L.mss_gated_workspace_bytes if isinstance(dims, mss.GatedDims) else L.mss_norm_workspace_bytes
    return f(ctypes.byref(dims), op, ctypes.byref(n)), n.value


# argument names and fake pointers of a valid call; outputs last
CALLS = {
    "mss_gated_scan": ["x", "r", "i", "decay", "z", "h0", "reset", "y", "h_ckpt", "h_last", "ws"],
    "mss_gated_scan_backward": ["x", "r", "i", "decay", "z", "reset", "h_ckpt", "dout", "dh_last", "dx", "dr", "di",
                                "ddecay", "dz", "dh0", "ws"],
    "mss_gated_step": ["x", "r", "i", "decay", "z", "h", "y"],
    "mss_add_norm": ["x", "residual", "w", "b", "scale", "s", "y"],
    "mss_add_norm_backward": ["s", "w", "dy", "ds", "x", "scale", "dx", "dresidual", "dw", "db", "dscale", "ws"],
    "mss_gated_norm": ["x", "z", "w", "b", "residual", "scale", "y"],
    "mss_gated_norm_backward": ["x", "z", "w", "b", "scale", "dout", "dx", "dz", "dw", "db", "dscale", "ws"],
}
OPS = {"mss_gated_scan": 4, "mss_gated_scan_backward": 5, "mss_add_norm_backward": 6, "mss_gated_norm_backward": 7}
OUTPUTS = {"mss_gated_scan": {"y", "h_ckpt", "h_last", "ws"},
           "mss_gated_scan_backward": {"dx", "dr", "di", "ddecay", "dz", "dh0", "ws"}, "mss_gated_step": {"h", "y"},
           "mss_add_norm": {"s", "y"}, "mss_add_norm_backward": {"dx", "dresidual", "dw", "db", "dscale", "ws"},
           "mss_gated_norm": {"y"}, "mss_gated_norm_backward": {"dx", "dz", "dw", "db", "dscale", "ws"}}
OPTIONAL = {"z", "h0", "reset", "h_ckpt", "h_last", "dh_last", "dh0", "residual", "b", "scale", "ds", "dx", "dw", "db",
            "dscale"}


def call(L, name, dims, st=None, ws_size=None, **over):
    args = {a: fake(i + 1) for i, a in enumerate(CALLS[name])}
    args.update(over)
    vals = list(args.values())
    if "ws" in args:
        vals.append(need(L, dims, OPS[name])[1] if ws_size is None else ws_size)
    return getattr(L, name)(ctypes.byref(dims) if dims is not None else None,
                            ctypes.byref(st) if st is not None else None, *vals, None)


def dims_of(name):
    return gated() if "gated_s" in name else norm(groups=1, order=0)


def refused(L, name, dims, **over):
    """The status of a call that would otherwise be valid: an aliasing output keeps it from
    ever launching, so a call wrongly accepted here reports EALIAS, not a launch."""
    outs = sorted(OUTPUTS[name] - {"ws"} - set(over))
    if not outs:                         # the one output is what is tried
        return call(L, name, dims, **over)
    out = outs[-1]
    inp = next(a for a in CALLS[name] if a not in OUTPUTS[name] and a not in over and a != "reset")
    args = {out: fake(CALLS[name].index(inp) + 1), **over}
    return call(L, name, dims, **args)


@pytest.mark.parametrize("name", CALLS)
def test_blocks_are_checked(L, name):
    assert call(L, name, None, ws_size=0) == EINVAL
    for field, value in (("struct_size", 8), ("flags", 1), ("dtype", 3), ("dtype", -1)):
        d = dims_of(name)
        setattr(d, field, value)
        assert refused(L, name, d, **({"ws_size": 1 << 30} if name in OPS else {})) == EINVAL, field
    st = strides(mss.GatedStrides if "gated_s" in name else mss.NormStrides, 64)
    for field, value in (("struct_size", 8), ("reserved", 1)):
        keep = getattr(st, field)
        setattr(st, field, value)
        assert refused(L, name, dims_of(name), st=st) == EINVAL, field
        setattr(st, field, keep)
    assert refused(L, name, dims_of(name)) == EALIAS                      # valid but for the overlap


@pytest.mark.parametrize("name", CALLS)
def test_pointers_are_checked(L, name):
    d = dims_of(name)
    sl = strides(mss.GatedStrides if "gated_s" in name else mss.NormStrides, 70)
    used = name in OPS and need(L, d, OPS[name])[1] > 0      # a call may need no workspace
    for i, a in enumerate(CALLS[name]):
        if a == "ws":
            if not used:
                continue
            assert call(L, name, d, ws=None) == EWORKSPACE
            assert call(L, name, d, ws_size=need(L, d, OPS[name])[1] - 1) == EWORKSPACE
            assert call(L, name, d, ws=fake(i + 1, 16)) == EALIGN
            continue
        if a not in OPTIONAL or (a == "dx" and name != "mss_add_norm_backward") or a == "h_ckpt" and "back" in name:
            assert refused(L, name, d, **{a: None}) == EINVAL, a
        if a != "reset":
            assert refused(L, name, d, **{a: fake(i + 1, 8)}) == EALIGN, a
        # with strides an activation needs its element's alignment only
        if a in ("x", "r", "i", "z", "y", "dout", "dx", "dy", "dresidual", "residual"):
            over = {a: fake(1, 2) if OUTPUTS[name] == {a} else fake(i + 1, 2)}
            assert refused(L, name, d, st=sl, **over) == EALIAS, a
            assert refused(L, name, d, st=sl, **{a: fake(i + 1, 1)}) == EALIGN, a
    # every output against every input and every other output
    for o in OUTPUTS[name]:
        for a in CALLS[name]:
            if a == o or "ws" in (a, o) and not used or (name, {a, o}) == ("mss_add_norm", {"s", "residual"}):
                continue
            assert call(L, name, d, **{o: fake(CALLS[name].index(a) + 1)}) == EALIAS, (o, a)


def test_residual_updated_in_place_is_the_one_overlap_allowed(L):
    """s may be the residual itself; shifted, or with another stride, it may not (and y never)."""
    at = CALLS["mss_add_norm"].index("residual") + 1
    d = norm(M=4, D=64)
    assert call(L, "mss_add_norm", d, s=fake(at), y=fake(1)) == EALIAS    # y on x is still seen
    assert call(L, "mss_add_norm", d, s=fake(at, 16)) == EALIAS
    st = strides(mss.NormStrides, 64)
    st.s = 80
    assert call(L, "mss_add_norm", d, st=st, s=fake(at)) == EALIAS


@pytest.mark.parametrize("field", ("x", "r", "i", "z", "y", "dx", "dr", "di", "dz"))
def test_gated_strides(L, field):
    st = strides(mss.GatedStrides, 64)
    setattr(st, field, 63)
    assert refused(L, "mss_gated_scan_backward", gated(), st=st) == EINVAL
    setattr(st, field, 1 << 61)
    assert refused(L, "mss_gated_scan_backward", gated(), st=st) == EINVAL


def test_columns_of_one_buffer_may_interleave(L):
    """Four gradients as neighbouring column ranges of one (M, 256) buffer pass the overlap
    check (the call is stopped by another fault); moved by one element they do not."""
    st = strides(mss.GatedStrides, 64)
    st.dx = st.dr = st.di = st.dz = 256
    parts = {k: fake(40, 2 * 64 * n) for n, k in enumerate(("dx", "dr", "di", "dz"))}
    name, d = "mss_gated_scan_backward", gated()
    assert call(L, name, d, st=st, ws=None, **parts) == EWORKSPACE
    parts["dr"] = fake(40, 2 * 63)
    assert call(L, name, d, st=st, ws=None, **parts) == EALIAS
    # wrapped into the next row
    parts["dr"], parts["dz"] = fake(40, 2 * 64), fake(40, 2 * 193)
    assert call(L, name, d, st=st, ws=None, **parts) == EALIAS


def test_gate_arguments(L):
    for name in ("mss_gated_scan", "mss_gated_scan_backward", "mss_gated_step"):
        for bad in (dict(gate=3), dict(gate=-1), dict(B=-1), dict(D=-1), dict(scale=0.0), dict(scale=-1.0),
                    dict(scale=float("inf")), dict(scale=float("nan")), dict(B=1 << 40, L=1 << 20, D=1 << 20)):
            if name == "mss_gated_step" and bad.get("L"):
                bad = dict(B=1 << 40, D=1 << 30)
            kw = dict(ws_size=1 << 40) if name in OPS else {}
            assert call(L, name, gated(**bad), **kw) == EINVAL, (name, bad)
        # i and decay belong to the decay gate alone
        for gate in (0, 2):
            over = dict(di=None, ddecay=None) if "back" in name else {}
            assert refused(L, name, gated(gate=gate), i=None, **over) == EINVAL
            assert refused(L, name, gated(gate=gate), decay=None, **over) == EINVAL
    d = gated(gate=0)
    free = dict(i=None, decay=None)
    assert refused(L, "mss_gated_scan_backward", d, di=None, **free) == EINVAL     # ddecay left
    assert refused(L, "mss_gated_scan_backward", d, ddecay=None, **free) == EINVAL
    assert refused(L, "mss_gated_scan_backward", gated(), dz=None) == EINVAL       # z without dz
    assert refused(L, "mss_gated_scan_backward", gated(), z=None) == EINVAL        # dz without z
    assert call(L, "mss_gated_scan", gated(L=-1), ws_size=0) == EINVAL


def test_limits(L):
    """Widths, groups and launches past what the kernels count in 32 bits."""
    w = mss.MAX_WIDTH
    assert need(L, gated(B=1, L=2, D=w), 4)[0] == 0 and need(L, gated(B=1, L=2, D=w + 1), 4)[0] == EINVAL
    assert call(L, "mss_gated_step", gated(B=1, D=w + 1)) == EINVAL
    assert need(L, norm(M=1, D=w), 6)[0] == 0 and need(L, norm(M=1, D=w + 1), 6)[0] == EINVAL
    assert need(L, norm(M=1, D=1 << 20, groups=1 << 20), 7)[0] == 0
    assert need(L, norm(M=1, D=1 << 21, groups=1 << 21), 7)[0] == EINVAL
    # 2^32 threads: 2^23 workgroups of 512, each 128 (forward) or 64 (backward) steps of a tile
    for op, steps in ((4, 128), (5, 64)):
        assert need(L, gated(B=1, L=steps * ((1 << 23) - 1), D=1), op)[0] == 0
        assert need(L, gated(B=1, L=steps * (1 << 23), D=1), op)[0] == EINVAL
    assert call(L, "mss_gated_step", gated(B=1 << 32, D=1)) == EINVAL


def test_norm_arguments(L):
    for name in ("mss_add_norm", "mss_add_norm_backward", "mss_gated_norm", "mss_gated_norm_backward"):
        kw = dict(ws_size=1 << 40) if name in OPS else {}
        for bad in (dict(kind=2), dict(kind=-1), dict(M=-1), dict(D=-1), dict(groups=0), dict(groups=3), dict(eps=0.0),
                    dict(eps=-1.0), dict(eps=float("inf")), dict(eps=float("nan")), dict(alpha=float("nan")),
                    dict(alpha=float("inf")), dict(order=2), dict(res=2), dict(M=1 << 40, D=1 << 30)):
            assert call(L, name, norm(**bad), **kw) == EINVAL, (name, bad)
        add = "add" in name
        # add_norm: one group, no gate order, residual of the type or fp32
        assert refused(L, name, norm(groups=2)) == (EINVAL if add else EALIAS)
        assert refused(L, name, norm(order=1)) == (EINVAL if add else EALIAS)
        assert refused(L, name, norm(res=0)) == (EALIAS if add else EINVAL)
    assert refused(L, "mss_gated_norm_backward", norm(), dz=None) == EINVAL
    assert refused(L, "mss_gated_norm_backward", norm(), z=None) == EINVAL
    # x is needed, and looked at, only for dscale
    at = CALLS["mss_add_norm_backward"].index("x") + 1
    assert refused(L, "mss_add_norm_backward", norm(), x=None) == EINVAL
    assert call(L, "mss_add_norm_backward", norm(), x=None, dscale=None, ws=None) == EWORKSPACE
    assert call(L, "mss_add_norm_backward", norm(), dx=fake(at), dscale=None, ws=None) == EWORKSPACE


def test_workspace_queries(L):
    for op in (4, 5):
        st, n = need(L, gated(), op)
        assert st == 0 and n % 256 == 0
        assert need(L, gated(B=0), op) == (0, 0) and need(L, gated(L=0), op) == (0, 0)
        assert need(L, gated(gate=7), op) == (EINVAL, 0)
        assert need(L, gated(B=1 << 40, L=1 << 20, D=1 << 20), op) == (EINVAL, 0)
    for op in (6, 7):
        st, n = need(L, norm(), op)
        assert st == 0 and n > 0 and n % 256 == 0
        assert need(L, norm(M=0), op) == (0, 0) and need(L, norm(D=0), op) == (0, 0)
        assert need(L, norm(groups=3), op) == (EINVAL, 0)
    for op in (0, 1, 3, 6, 7):
        assert need(L, gated(), op)[0] == EINVAL
    for op in (1, 4, 5):
        assert need(L, norm(), op)[0] == EINVAL
    assert L.mss_gated_workspace_bytes(ctypes.byref(gated()), 4, None) == EINVAL
    assert L.mss_norm_workspace_bytes(ctypes.byref(norm()), 6, None) == EINVAL
    # the binding asks for the same
    assert mss.gated_workspace_bytes(mss.OP_GATED_SCAN_BACKWARD, batch=2, seq_len=100, d_inner=64,
                                     gate="decay") == need(L, gated(), 5)[1]
    assert mss.norm_workspace_bytes(mss.OP_ADD_NORM_BACKWARD, rows=10, width=64) == need(L, norm(), 6)[1]


@pytest.mark.parametrize("name", CALLS)
def test_empty_problems_launch_nothing(L, name):
    d = gated(B=0) if "gated_s" in name else norm(M=0)
    keep = {"decay", "w", "ddecay"}      # still hold a value per channel
    over = {a: None for a in CALLS[name] if a not in keep}
    if "ddecay" in CALLS[name]:
        assert call(L, name, d, **{**over, "ddecay": None}) == EINVAL
        return                           # its zeroing would launch
    assert call(L, name, d, **over) == 0
    d = gated(D=0) if "gated_s" in name else norm(D=0)
    assert call(L, name, d, **{a: None for a in CALLS[name]}) == 0
