"""Refusals of the embedding, the head's loss and clipping at the C ABI, without a GPU: every call
is rejected, or is empty, before any launch, so the pointers are fake addresses that are never
dereferenced."""
from __future__ import annotations

import ctypes

import pytest

import mamba_selective_scan_causal_amd as mss

OK, EINVAL, EALIGN, EALIAS, EWORKSPACE = 0, -1, -2, -3, -4
BASE = 0x7F0000000000


def fake(i, off=0):
    return ctypes.c_void_p(BASE + i * (1 << 32) + off)


@pytest.fixture(scope="module")
def L():
    return mss.lib()


def embed(M=10, V=100, D=64, dtype=1, out=1, ids=8, scale=1.0, flags=0):
    return mss.EmbedDims(ctypes.sizeof(mss.EmbedDims), flags, dtype, out, ids, 0, M, V, D, scale, 0)


def head(M=10, V=100, D=64, dtype=1, ids=8, scale=1.0):
    return mss.HeadDims(ctypes.sizeof(mss.HeadDims), 0, dtype, ids, M, V, D, scale, 0)


CALLS = {
    "mss_embedding": ["ids", "weight", "y"],
    "mss_embedding_backward": ["ids", "dy", "dweight", "ws"],
    "mss_head_loss": ["x", "weight", "targets", "loss", "lse", "ws"],
    "mss_head_loss_backward": ["x", "weight", "targets", "lse", "dloss", "dlse", "dx", "dweight", "ws"],
}
OUTPUTS = {"mss_embedding": {"y"}, "mss_embedding_backward": {"dweight", "ws"}, "mss_head_loss": {"loss", "lse", "ws"},
           "mss_head_loss_backward": {"dx", "dweight", "ws"}}
OPTIONAL = {"mss_head_loss_backward": {"dlse", "dx", "dweight"}}


def dims_of(name, **kw):
    return (embed if "embed" in name else head)(**kw)


def need(L, name, dims):
    n = ctypes.c_size_t(0)
    if "embed" in name:
        st = L.mss_embed_workspace_bytes(ctypes.byref(dims), ctypes.byref(n))
    else:
        st = L.mss_head_workspace_bytes(ctypes.byref(dims), 9 if "backward" in name else 8, ctypes.byref(n))
    return st, n.value


def call(L, name, dims, st=None, ws_size=None, **over):
    args = {a: fake(i + 1) for i, a in enumerate(CALLS[name])}
    args.update(over)
    vals = list(args.values())
    if "ws" in args:
        vals.append(need(L, name, dims)[1] if ws_size is None else ws_size)
    return getattr(L, name)(ctypes.byref(dims) if dims is not None else None,
                            ctypes.byref(st) if st is not None else None, *vals, None)


def refused(L, name, dims, st=None, **over):
    """The status of a call that would be valid but for what is tried: an output on an input keeps
    it from ever launching, so a call wrongly accepted here reports EALIAS."""
    out = next(o for o in CALLS[name] if o in OUTPUTS[name] and o not in over and o != "ws") if set(
        OUTPUTS[name]) - {"ws"} - set(over) else None
    inp = next(a for a in CALLS[name] if a not in OUTPUTS[name] and a not in over)
    if out:
        over[out] = fake(CALLS[name].index(inp) + 1)
    return call(L, name, dims, st, **over)


@pytest.mark.parametrize("name", CALLS)
def test_blocks_are_checked(L, name):
    ws = {"ws_size": 1 << 50} if "ws" in CALLS[name] else {}
    assert call(L, name, None, **({"ws_size": 0} if ws else {})) == EINVAL
    bad = [("struct_size", 8), ("flags", 2), ("flags", -1), ("dtype", 3), ("dtype", -1), ("id_bytes", 2),
           ("id_bytes", 0), ("rows", -1), ("vocab", -1), ("width", -1), ("rows", 1 << 26), ("vocab", 1 << 26),
           ("width", (1 << 28) + 1), ("reserved", 1)]
    if "embed" in name:
        bad += [("out_dtype", 2), ("out_dtype", 5), ("scale", float("nan")), ("scale", float("inf")), ("reserved2", 1)]
        if "backward" not in name:
            bad += [("flags", 1)]
    else:
        bad += [("logit_scale", float("inf")), ("vocab", 0), ("width", 0)]
    for field, value in bad:
        d = dims_of(name)
        setattr(d, field, value)
        assert refused(L, name, d, **ws) == EINVAL, (field, value)
    cls = mss.EmbedStrides if "embed" in name else mss.HeadStrides
    for field, value in (("struct_size", 4), ("reserved", 1)):
        st = cls(*([64] * len(cls._fields_)))
        st.struct_size, st.reserved = ctypes.sizeof(cls), 0
        setattr(st, field, value)
        assert refused(L, name, dims_of(name), st, **ws) == EINVAL, field
    assert refused(L, name, dims_of(name)) == EALIAS                 # the rest was in order


@pytest.mark.parametrize("name", CALLS)
def test_required_tensors(L, name):
    for a in CALLS[name]:
        if a == "ws" or a in OPTIONAL.get(name, ()):
            continue
        assert refused(L, name, dims_of(name), **{a: None}) == EINVAL, a


@pytest.mark.parametrize("name", CALLS)
def test_strides_below_the_width(L, name):
    cls = mss.EmbedStrides if "embed" in name else mss.HeadStrides
    fields = [f for f, _ in cls._fields_[2:]]
    if name == "mss_head_loss":
        fields = ["x", "weight"]
    for f in fields:
        st = cls(ctypes.sizeof(cls), 0, *([64] * (len(cls._fields_) - 2)))
        setattr(st, f, 63)
        assert refused(L, name, dims_of(name), st) == EINVAL, f
        setattr(st, f, 1 << 62)
        assert refused(L, name, dims_of(name), st) == EINVAL, f


@pytest.mark.parametrize("name", CALLS)
def test_alignment(L, name):
    per_row = {"ids", "targets", "loss", "lse", "dloss", "dlse"}
    cls = mss.EmbedStrides if "embed" in name else mss.HeadStrides
    st = cls(ctypes.sizeof(cls), 0, *([72] * (len(cls._fields_) - 2)))
    for i, a in enumerate(CALLS[name]):
        if OUTPUTS[name] - {"ws"} == {a}:
            i = 0                                    # the one output: on the first input
        if a == "ws":
            assert call(L, name, dims_of(name), ws=fake(20, 128)) == EALIGN
            continue
        if a in per_row:
            assert refused(L, name, dims_of(name), **{a: fake(i + 1, 2)}) == EALIGN, a
            assert refused(L, name, dims_of(name, ids=4), **{a: fake(i + 1, 4)}) == EALIAS, a
            continue
        assert refused(L, name, dims_of(name), **{a: fake(i + 1, 8)}) == EALIGN, a        # dense: 16 bytes
        assert refused(L, name, dims_of(name), st, **{a: fake(i + 1, 1)}) == EALIGN, a
        assert refused(L, name, dims_of(name), st, **{a: fake(i + 1, 2)}) == EALIAS, a


@pytest.mark.parametrize("name", CALLS)
def test_outputs_overlap_nothing(L, name):
    for out in OUTPUTS[name]:
        for a in CALLS[name]:
            if a == out:
                continue
            assert call(L, name, dims_of(name), **{out: fake(CALLS[name].index(a) + 1)}) == EALIAS, (out, a)


@pytest.mark.parametrize("name", [n for n in CALLS if "ws" in CALLS[n]])
def test_workspace(L, name):
    st, n = need(L, name, dims_of(name))
    assert st == OK and n > 0
    assert call(L, name, dims_of(name), ws=None) == EWORKSPACE
    assert call(L, name, dims_of(name), ws_size=n - 1) == EWORKSPACE
    assert L.mss_head_workspace_bytes(ctypes.byref(head()), 7, ctypes.byref(ctypes.c_size_t(0))) == EINVAL
    # a function of the sizes: more rows never need less
    last = 0
    for M in (0, 1, 100, 1000, 10000, 100000):
        st, n = need(L, name, dims_of(name, M=M))
        assert st == OK and n >= last or "head" in name
        last = n


def test_sizes_that_fit_no_launch(L):
    big = (1 << 26) - 1
    assert need(L, "mss_head_loss_backward", head(M=big, V=big, D=1 << 28))[0] == EINVAL
    assert need(L, "mss_embedding_backward", embed(M=big, V=big, D=1 << 28))[0] == EINVAL
    assert call(L, "mss_embedding_backward", embed(M=big, V=big, D=1 << 28), ws_size=1 << 60) == EINVAL


def test_empty_calls(L):
    assert L.mss_embedding(ctypes.byref(embed(M=0)), None, None, fake(1), None, None) == OK
    assert L.mss_embedding(ctypes.byref(embed(D=0)), None, fake(1), None, None, None) == OK
    assert call(L, "mss_embedding_backward", embed(V=0), dweight=None) == OK
    assert call(L, "mss_embedding_backward", embed(M=0, flags=1)) == OK
    assert call(L, "mss_head_loss", head(M=0)) == OK
    assert call(L, "mss_head_loss_backward", head(), dx=None, dweight=None) == OK
    assert call(L, "mss_head_loss_backward", head(M=0), dweight=None) == OK


def tensors(*rows):
    return (mss.ListTensor * len(rows))(*[(p.value if p else None, o.value if o else None, n, t, u)
                                          for p, o, n, t, u in rows])


def clip(L, rows, scale=1.0, max_norm=1.0, norm=fake(90), ws=fake(91), size=1 << 40, count=None, f="clip"):
    t = tensors(*rows)
    n = len(rows) if count is None else count
    if f == "clip":
        return L.mss_clip_grads(t, n, scale, max_norm, norm, ws, size, None)
    return L.mss_grad_norm(t, n, scale, norm, ws, size, None)


def test_lists(L):
    good = (fake(1), fake(1), 100, 1, 1)
    clash = (fake(3), fake(3), 8, 0, 0)
    # every call below has two tensors in one place, so that none is ever launched
    assert clip(L, [good, clash, clash]) == EALIAS
    bad = [((None, fake(1), 100, 1, 1), EINVAL), ((fake(1), None, 100, 1, 1), EINVAL), ((fake(1), fake(1), -1, 1, 1), EINVAL),
           ((fake(1), fake(1), 1 << 44, 1, 1), EINVAL), ((fake(1), fake(1), 100, 3, 3), EINVAL),
           ((fake(1), fake(2), 100, 0, 1), EINVAL), ((fake(1), fake(2), 100, 1, 2), EINVAL),
           ((fake(1, 1), fake(2), 100, 1, 1), EALIGN), ((fake(1), fake(2, 2), 100, 1, 0), EALIGN)]
    for t, status in bad:
        assert clip(L, [t, clash, clash]) == status, t
    assert clip(L, [(fake(1), fake(1), 1 << 43, 1, 1), (fake(2), fake(2), 1 << 43, 1, 1), clash, clash]) == EINVAL
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(max_norm=-1.0),
               dict(max_norm=float("inf")), dict(norm=None), dict(count=-1), dict(count=1 << 31)):
        assert clip(L, [good, clash, clash], **kw) == EINVAL, kw
    assert clip(L, [good, clash, clash], norm=fake(90, 2)) == EALIGN
    assert clip(L, [good], ws=None) == EWORKSPACE and clip(L, [good], size=100) == EWORKSPACE
    assert clip(L, [good], ws=fake(91, 16)) == EALIGN
    assert L.mss_clip_grads(None, 1, 1.0, 1.0, fake(90), fake(91), 1 << 40, None) == EINVAL


def test_lists_overlap_nothing(L):
    t = lambda p, o, n=100: (p, o, n, 1, 1)
    for rows in ([t(fake(1), fake(1)), t(fake(1, 100), fake(1, 100))],         # two in place
                 [t(fake(1), fake(2)), t(fake(2, 198), fake(3))],              # one's output, another's input
                 [t(fake(1), fake(2)), t(fake(3), fake(2, 198))],              # two outputs
                 [t(fake(1), fake(1, 2))],                                     # nearly in place
                 [(fake(1), fake(1), 100, 1, 0)],                              # in place, but wider
                 [t(fake(1), fake(1)), t(fake(90), fake(90))],                 # the norm
                 [t(fake(91), fake(91))]):                                     # the workspace
        assert clip(L, rows) == EALIAS, rows
    assert clip(L, [t(fake(90), None)], f="norm") == EALIAS
    # inputs may lie anywhere: the workspace is what is wrong here
    assert clip(L, [t(fake(1), fake(2)), t(fake(1), fake(3)), t(fake(1, 4), fake(4))], size=1) == EWORKSPACE
    assert clip(L, [t(fake(1), fake(1)), t(fake(1, 200), fake(1, 200))], size=1) == EWORKSPACE     # neighbours


def test_structs_are_laid_out_as_the_header_says():
    assert ctypes.sizeof(mss.EmbedDims) == 56 and ctypes.sizeof(mss.EmbedStrides) == 24
    assert ctypes.sizeof(mss.HeadDims) == 48 and ctypes.sizeof(mss.HeadStrides) == 40
    assert ctypes.sizeof(mss.ListTensor) == 32
