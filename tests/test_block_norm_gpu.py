"""The norms before and after a block on the GPU, forward and backward, against
the fp64 forms of block_ref within their derived bounds."""
from __future__ import annotations

import numpy as np
import pytest

import block_ref as ref
import mamba_selective_scan_causal_amd as mss
from block_util import back, check, column_slice, outside_is_nan, put, torch_type
from gpu_util import announce

pytestmark = pytest.mark.gpu

EPS = 1e-6


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


def add_case(M, D, dtype, res, kind, *, residual=True, scale=True, bias=True, ds=True, seed=0, spread=1.0):
    import torch
    rng = np.random.default_rng(seed + 31 * M + D)
    n = lambda *s: rng.normal(size=s)
    x, dy = put(spread * n(M, D), dtype), put(n(M, D), dtype)
    old = put(spread * 2 * n(M, D) + 0.5, res) if residual else None
    up = put(n(M, D), res) if ds else None
    w, b = put(1 + 0.2 * n(D)), put(n(D)) if bias else None
    sc = put(1 + 0.2 * n(D)) if scale else None
    kw = dict(kind=kind, eps=EPS, alpha=0.7)
    y, s = mss.add_norm(x, old, w, b, sc, res_dtype=torch_type(res), **kw)
    g = mss.add_norm_backward(s, w, dy, up, x if scale else None, sc, bias=bias, **kw)
    torch.cuda.synchronize()
    assert s.dtype == torch_type(res) and y.dtype == x.dtype
    hs, hw = back(s), back(w)
    want, bound = ref.add_norm(back(x), back(old), back(sc), 0.7)
    worst = {"s": check(s, want, bound, res, "s")}
    want, bound = ref.norm_of(hs, hw, back(b), kind, EPS)
    worst["y"] = check(y, want, bound, dtype, "y")
    val, tol = ref.add_norm_backward(hs, hw, back(dy), back(up), back(x) if scale else None, back(sc),
                                     kind=kind, eps=EPS, alpha=0.7)
    for k, v in g.items():
        if v is None:
            assert k in ("dbias", "dscale")
            continue
        t = dtype if k == "dx" else res if k == "dresidual" else "f32"
        worst[k] = check(v, val[k], tol[k], t, k)
    announce(f"M{M} D{D} {dtype}/{res} {kind} worst " + " ".join(f"{k}={v:.2f}" for k, v in worst.items()))


def gated_case(M, D, dtype, kind, order, groups=1, *, z=True, residual=True, scale=True, bias=True, seed=0,
               spread=1.0):
    import torch
    rng = np.random.default_rng(seed + 17 * M + D)
    n = lambda *s: rng.normal(size=s)
    x, dout = put(spread * (n(M, D) + 0.3), dtype), put(n(M, D), dtype)
    zt = put(n(M, D), dtype) if z else None
    old = put(n(M, D), dtype) if residual else None
    w, b = put(1 + 0.2 * n(D)), put(n(D)) if bias else None
    sc = put(1 + 0.2 * n(D)) if scale else None
    kw = dict(groups=groups, order=order, kind=kind, eps=EPS, alpha=0.7)
    y = mss.gated_norm(x, zt, w, b, old, sc, **kw)
    g = mss.gated_norm_backward(x, zt, w, b, sc, dout, **kw)
    torch.cuda.synchronize()
    val, tol = ref.gated_norm(*(back(t) for t in (x, zt, w, b, old, sc, dout)), **kw)
    worst = {"y": check(y, val["y"], tol["y"], dtype, "y")}
    for k, v in g.items():
        if v is not None:
            worst[k] = check(v, val[k], tol[k], dtype if k in ("dx", "dz") else "f32", k)
    assert (g["dz"] is None) == (not z)
    announce(f"M{M} D{D} {dtype} {kind} {order} g{groups} worst " + " ".join(f"{k}={v:.2f}" for k, v in worst.items()))


TYPE_PAIRS = (("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"))
# widths around a wave, a workgroup and their vector pieces, odd ones, one channel, a wide row
SIZES = [(1, 1), (2, 7), (3, 64), (5, 65), (33, 100), (2, 127), (1, 128), (9, 255), (4, 256), (130, 257), (3, 513),
         (17, 768), (2, 1001), (5, 1024), (3, 1536), (2, 2050), (4, 2560), (700, 40), (3, 4097), (2, 5120), (1, 9000),
         (2, 16384), (1, 40001)]


@pytest.mark.parametrize("dtype,res", TYPE_PAIRS)
@pytest.mark.parametrize("kind", ("rms", "layer"))
def test_add_norm_types(dtype, res, kind):
    add_case(70, 520, dtype, res, kind)
    add_case(3, 333, dtype, res, kind, residual=False, scale=False, bias=False, ds=False)


@pytest.mark.parametrize("M,D", SIZES)
def test_add_norm_sizes(M, D):
    add_case(M, D, "bf16", "f32", "rms", bias=False)
    add_case(M, D, "f32", "f32", "layer", scale=D % 2 == 0)
    add_case(M, D, "f16", "f16", "layer", scale=D % 2 == 1, ds=False)


@pytest.mark.parametrize("dtype", ("f32", "bf16", "f16"))
@pytest.mark.parametrize("kind", ("rms", "layer"))
@pytest.mark.parametrize("order", ("before", "after"))
def test_gated_norm_types(dtype, kind, order):
    gated_case(70, 520, dtype, kind, order, 4)
    gated_case(3, 333, dtype, kind, order, 3, residual=False, scale=False, bias=False)
    gated_case(5, 96, dtype, kind, order, z=False)


@pytest.mark.parametrize("M,D", SIZES)
def test_gated_norm_sizes(M, D):
    gated_case(M, D, "bf16", "rms", "before", residual=False, scale=False, bias=False)
    gated_case(M, D, "f32", "layer", "after")
    gated_case(M, D, "f16", "rms", "after", bias=False)


# groups of one channel, of odd widths, of a wave, wider than a wave, many of them
@pytest.mark.parametrize("D,groups", [(8, 8), (21, 3), (80, 16), (128, 2), (520, 8), (1536, 8), (1998, 2), (5120, 8),
                                      (5120, 80), (6150, 6), (12000, 3)])
@pytest.mark.parametrize("order", ("before", "after"))
def test_gated_norm_groups(D, groups, order):
    gated_case(19, D, "bf16", "rms", order, groups, residual=order == "after")
    gated_case(6, D, "f32", "layer" if D > groups else "rms", order, groups)


@pytest.mark.parametrize("res", ("f32", "f16"))
@pytest.mark.parametrize("D", (1001, 17000))
def test_stream_rounds_as_scale_and_add_do(res, D):
    """s is the product's rounding added and rounded, bit for bit: in a half-precision stream with
    a scale of 0.7 one sum in sixty lies next to a tie, which a fused product breaks otherwise."""
    import torch
    rng = np.random.default_rng(8)
    x, old, w = put(rng.normal(size=(40, D)), "f16"), put(2 * rng.normal(size=(40, D)), res), put(np.ones(D))
    sc = put(1 + 0.2 * rng.normal(size=D))
    for scale, k in ((None, 0.7), (sc, 0.7 * sc)):
        _, s = mss.add_norm(x, old, w, scale=scale, alpha=0.7)
        want = (old.float() + k * x.float()).to(old.dtype)
        torch.cuda.synchronize()
        assert torch.equal(s, want)


def test_many_rows():
    add_case(5001, 96, "bf16", "f32", "rms")
    gated_case(5001, 96, "bf16", "rms", "before", 2)


@pytest.mark.parametrize("kind", ("rms", "layer"))
def test_large_and_small_values(kind):
    """Rows far from 1: the squares of 1e15 and 1e-15 stay inside fp32 after the mean."""
    for spread in (1e15, 1e-12):
        add_case(4, 300, "f32", "f32", kind, bias=False, ds=False, scale=False, spread=spread)
        gated_case(4, 300, "f32", kind, "after", residual=False, spread=spread)


def test_rows_of_zeros_and_constants():
    """A row of zeros (padding) has norm 0, not NaN, and a gradient of g w / sqrt(eps); a constant row has
    layer norm 0 to within what its mean is known to."""
    import torch
    x = torch.zeros((3, 200), device="cuda")
    x[1] = 3.0
    w = torch.ones(200, device="cuda")
    for kind in ("rms", "layer"):
        y, s = mss.add_norm(x, None, w, kind=kind, eps=1e-4)
        g = mss.add_norm_backward(s, w, torch.ones_like(x), kind=kind, eps=1e-4)
        n = mss.gated_norm(x, x, w, kind=kind, eps=1e-4)
        torch.cuda.synchronize()
        assert torch.equal(y[0], x[0]) and torch.equal(n[0], x[0])
        assert all(torch.isfinite(t).all() for t in (y, s, n, g["dx"], g["dweight"]))
        want = 100.0 if kind == "rms" else 0.0
        assert torch.allclose(g["dx"][0], torch.full_like(x[0], want), rtol=1e-5, atol=1e-3)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("D", (96, 101, 2052))
def test_column_slices(dtype, D):
    """Strided rows give the dense call's bits and write nothing outside their columns."""
    import torch
    rng = np.random.default_rng(3)
    M = 37
    x, z, res, dout = (put(rng.normal(size=(M, D)), dtype) for _ in range(4))
    w, b, sc = (put(rng.normal(size=D)) for _ in range(3))
    sl = lambda t, o: column_slice(t, 5, o)[0]
    blank = lambda: column_slice(torch.full_like(x, float("nan")))
    kw = dict(order="after", alpha=0.5)
    y = mss.gated_norm(x, z, w, b, res, sc, **kw)
    g = mss.gated_norm_backward(x, z, w, b, sc, dout, **kw)
    (o, ow), (dx, dxw), (dz, dzw) = blank(), blank(), blank()
    mss.gated_norm(sl(x, 1), sl(z, 2), w, b, sl(res, 3), sc, out=o, **kw)
    g2 = mss.gated_norm_backward(sl(x, 1), sl(z, 2), w, b, sc, sl(dout, 1), out=dict(dx=dx, dz=dz), **kw)
    torch.cuda.synchronize()
    assert torch.equal(o, y) and all(outside_is_nan(t, D) for t in (ow, dxw, dzw))
    for k in g:
        assert torch.equal(g[k], g2[k]), k
    y, s = mss.add_norm(x, res, w, b, sc)
    g = mss.add_norm_backward(s, w, dout, res, x, sc, bias=True)
    (o, ow), (s2, sw), (dx, dxw), (dr, drw) = blank(), blank(), blank(), blank()
    mss.add_norm(sl(x, 2), sl(res, 1), w, b, sc, out=o, residual_out=s2)
    g2 = mss.add_norm_backward(s2, w, sl(dout, 3), sl(res, 1), sl(x, 2), sc, bias=True,
                               out=dict(dx=dx, dresidual=dr))
    torch.cuda.synchronize()
    assert torch.equal(o, y) and torch.equal(s2, s)
    assert all(outside_is_nan(t, D) for t in (ow, sw, dxw, drw))
    for k in g:
        assert torch.equal(g[k], g2[k]), k


@pytest.mark.parametrize("D", (96, 1001, 30000))
def test_residual_in_place(D):
    import torch
    rng = np.random.default_rng(4)
    x, res = put(rng.normal(size=(9, D)), "bf16"), put(rng.normal(size=(9, D)))
    w = put(rng.normal(size=D))
    y, s = mss.add_norm(x, res, w)
    stream = res.clone()
    y2, s2 = mss.add_norm(x, stream, w, residual_out=stream)
    torch.cuda.synchronize()
    assert s2 is stream and torch.equal(s, s2) and torch.equal(y, y2)


@pytest.mark.parametrize("dtype", ("bf16", "f32"))
@pytest.mark.parametrize("M,D", [(5000, 121), (700, 509), (3000, 1027), (600, 2561), (40, 8197)])
def test_residual_in_place_at_odd_widths(dtype, M, D):
    """A row's end is read together with channels of the lane before, which may
    have written its own already."""
    import torch
    rng = np.random.default_rng(D)
    x, res = put(rng.normal(size=(M, D)), dtype), put(rng.normal(size=(M, D)), dtype)
    w, b = put(rng.normal(size=D)), put(rng.normal(size=D))
    for kind in ("rms", "layer"):
        y, s = mss.add_norm(x, res, w, b, kind=kind)
        assert torch.equal(s, (res.float() + x.float()).to(s.dtype))
        for _ in range(3):
            stream = res.clone()
            y2, _ = mss.add_norm(x, stream, w, b, kind=kind, residual_out=stream)
            assert torch.equal(s, stream) and torch.equal(y, y2)


# every length of a last vector, in each team: 16 lanes, a wave, workgroups of
# some waves whose last has one lane, workgroups with two vectors a lane
@pytest.mark.parametrize("D", [*range(1, 18), 121, 127, 129, 130, 135, 509, 511, 513, 515, 517, 518, 1023, 2562,
                               4091, 4099, 8190, 8193, 8199, 12281])
@pytest.mark.parametrize("dtype", ("f16", "bf16", "f32"))
def test_row_ends(dtype, D):
    kind = ("rms", "layer")[D % 2]
    add_case(37, D, dtype, dtype if D % 3 else "f32", kind, seed=D)
    gated_case(37, D, dtype, kind, ("before", "after")[D % 3 > 0], seed=D)


@pytest.mark.parametrize("D,groups", [(286, 2), (1001, 7), (1030, 2), (2050, 5), (16394, 2), (20, 4), (22, 2)])
@pytest.mark.parametrize("dtype", ("f16", "f32"))
def test_group_ends(dtype, D, groups):
    """Group ends inside a row: the channels read before and after them are
    another group's."""
    gated_case(29, D, dtype, "layer", "before", groups, seed=groups)
    gated_case(29, D, dtype, "rms", "after", groups, seed=groups)


def test_empty():
    import torch
    f = dict(device="cuda")
    for M, D in ((0, 40), (3, 0)):
        x, w = torch.empty((M, D), **f), torch.ones(D, **f)
        y, s = mss.add_norm(x, x, w)
        g = mss.add_norm_backward(s, w, x, x, x, w, bias=True)
        n = mss.gated_norm(x, x, w, w, x, w)
        h = mss.gated_norm_backward(x, x, w, w, w, x)
        torch.cuda.synchronize()
        assert y.shape == s.shape == n.shape == (M, D)
        for t in (g["dweight"], g["dbias"], g["dscale"], h["dweight"], h["dbias"], h["dscale"]):
            assert t.shape == (D,) and not t.any()


def test_only_what_is_asked_for():
    import torch
    rng = np.random.default_rng(5)
    s, dy = put(rng.normal(size=(20, 300))), put(rng.normal(size=(20, 300)))
    w = put(rng.normal(size=300))
    full = mss.add_norm_backward(s, w, dy, bias=True)
    part = mss.add_norm_backward(s, w, dy, need_dx=False)
    torch.cuda.synchronize()
    assert part["dx"] is None and part["dbias"] is None and part["dscale"] is None
    assert torch.equal(part["dresidual"], full["dresidual"]) and torch.equal(part["dweight"], full["dweight"])
    assert torch.equal(full["dx"], full["dresidual"])


def test_binding_refuses():
    import torch
    x, w = torch.zeros((4, 8), device="cuda"), torch.ones(8, device="cuda")
    with pytest.raises(ValueError, match="kind must be"):
        mss.add_norm(x, None, w, kind="batch")
    with pytest.raises(ValueError, match="order must be"):
        mss.gated_norm(x, x, w, order="around")
    with pytest.raises(TypeError, match="residual stream must be"):
        mss.add_norm(x, x.bfloat16(), w)
    with pytest.raises(ValueError, match="expected shape"):
        mss.add_norm(x, x[:2], w)
    with pytest.raises(ValueError, match="weight is required"):
        mss.gated_norm(x, x, None)
    with pytest.raises(ValueError, match="x is required"):
        mss.add_norm_backward(x, w, x, scale=w)
    with pytest.raises(ValueError, match="contiguous"):
        mss.add_norm(x, None, torch.ones(16, device="cuda")[::2])
    for bad in (dict(groups=3), dict(eps=0.0), dict(alpha=float("nan")), dict(groups=0)):
        with pytest.raises(mss.MssError) as err:
            mss.gated_norm(x, x, w, **bad)
        assert err.value.status == -1
    with pytest.raises(mss.MssError) as err:
        mss.gated_norm(x, x, w, out=x)
    assert err.value.status == -3
