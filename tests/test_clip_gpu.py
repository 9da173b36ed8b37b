"""The norm of a list of gradients and clipping by it, against float64."""
from __future__ import annotations

import pytest
import torch

import ends_ref as ref
import mamba_selective_scan_causal_amd as mss
from ends_util import TYPES, check, generator, normal
from gpu_util import announce

pytestmark = pytest.mark.gpu

LISTS = {
    "one": [("f32", (1,))],
    "odd": [("bf16", (7, 9)), ("f16", (1001,)), ("f32", (3, 5, 2)), ("bf16", (1,))],
    "chunk ends": [("f32", (16383,)), ("bf16", (16384,)), ("f16", (16385,)), ("f32", (32768 + 7,))],
    "many": [(("f32", "bf16", "f16")[k % 3], (k + 1,)) for k in range(300)],
    "empty ones": [("f32", (0,)), ("bf16", (40, 0)), ("bf16", (33,)), ("f32", (0, 3))],
    "large": [("bf16", (3000, 1111)), ("f32", (517, 800))],
}


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


def tensors(name, std=1.0):
    g = generator(len(name))
    return [normal(g, *shape, std=std * (1 + k % 4), dtype=TYPES[t]) for k, (t, shape) in enumerate(LISTS[name])]


@pytest.mark.parametrize("name", LISTS)
@pytest.mark.parametrize("scale,max_norm", [(1.0, 1.0), (0.125, 1e6), (3.0, 0.5), (1.0, 0.0)])
@pytest.mark.parametrize("where", ["in place", "same types", "f32"])
def test_clip(name, scale, max_norm, where):
    grads = tensors(name)
    types = [g.dtype if where != "f32" else torch.float32 for g in grads]
    (norm, off), outs = ref.clip(grads, max_norm, scale, types)
    here = [g.cuda() for g in grads]
    to = None if where == "in place" else [torch.full(g.shape, 7.0, dtype=t, device="cuda") for g, t in zip(grads, types)]
    n0 = mss.grad_norm(here, scale=scale)
    got, n = mss.clip_grads(here, max_norm, scale=scale, out=to)
    torch.cuda.synchronize()
    assert n.shape == () and torch.equal(n, n0) and abs(n.item() - norm) <= off
    for k, (o, want) in enumerate(zip(got, outs)):
        assert o.dtype == types[k]
        check(o, want, f"{name}[{k}]")
        if where != "in place":
            assert torch.equal(here[k].cpu(), grads[k])


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_norm_that_is_not_finite_leaves_everything(bad):
    grads = [g.cuda() for g in tensors("odd")]
    grads[1][13] = bad
    kept = [g.clone() for g in grads]
    out, norm = mss.clip_grads(grads, 1.0, scale=0.5)
    assert not torch.isfinite(norm)
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert all(same(a, b) for a, b in zip(grads, kept))
    to, _ = mss.clip_grads(grads, 1.0, scale=0.5, out=[torch.zeros_like(g) for g in grads])
    assert all(torch.equal(torch.nan_to_num(a, 5), torch.nan_to_num(b, 5)) for a, b in zip(to, kept))


def test_squares_do_not_overflow_or_vanish():
    for v, n in ((1e30, 1e30 * 1000 ** 0.5), (1e-30, 1e-30 * 1000 ** 0.5)):
        g = torch.full((1000,), v, device="cuda")
        got = mss.grad_norm([g]).item()
        assert abs(got / (n / v * g[0].double().item()) - 1) <= 4 * ref.U
    out, norm = mss.clip_grads([torch.full((1000,), 1e30, device="cuda")], 1.0)
    assert torch.allclose(out[0], torch.full((1000,), 1000 ** -0.5, device="cuda"), rtol=1e-6)
    # a norm beyond fp32 is reported as infinite; the tensors are clipped by the norm itself
    big = torch.full((100000,), 3e38, device="cuda")
    out, norm = mss.clip_grads([big], 1.0)
    assert torch.isinf(norm) and torch.allclose(out[0], torch.full_like(big, 100000 ** -0.5), rtol=1e-6)


def test_views_of_one_buffer():
    """Neighbouring views at any alignment: each value once, the bytes between them left alone."""
    g = generator(3)
    flat = normal(g, 5000, dtype=torch.bfloat16).cuda()
    kept = flat.clone()
    at = [(1, 700), (701, 33), (735, 1), (737, 4001)]
    grads = [flat[a:a + n] for a, n in at]
    (norm, off), outs = ref.clip([v.cpu() for v in grads], 2.0, 1.0, [torch.bfloat16] * 4)
    got, n = mss.clip_grads(grads, 2.0)
    assert abs(n.item() - norm) <= off
    for o, want in zip(got, outs):
        check(o, want, "view")
    outside = torch.ones(5000, dtype=torch.bool)
    for a, m in at:
        outside[a:a + m] = False
    assert torch.equal(flat.cpu()[outside], kept.cpu()[outside])


def test_gradients_that_are_none():
    g = [None, torch.full((4,), 3.0, device="cuda"), None]
    out, norm = mss.clip_grads(g, 3.0)
    assert out[0] is None and out[2] is None and norm.item() == 6.0 and (out[1] == 1.5).all()
    assert mss.grad_norm(g, scale=2.0).item() == 6.0


def test_some_in_place_some_not():
    a, b = torch.full((40,), 2.0, device="cuda"), torch.full((24,), 2.0, device="cuda")
    to = torch.zeros(24, device="cuda")
    out, norm = mss.clip_grads([a, b], 8.0, out=[a, to])
    assert norm.item() == 16.0 and (a == 1).all() and (b == 2).all() and (to == 1).all()


def test_refusals():
    g = torch.ones(10, device="cuda")
    with pytest.raises(ValueError):
        mss.clip_grads([], 1.0)
    with pytest.raises(ValueError):
        mss.clip_grads([None], 1.0)
    with pytest.raises(TypeError):
        mss.grad_norm([g.double()])
    with pytest.raises(TypeError):
        mss.grad_norm([g, 3])
    with pytest.raises(ValueError):
        mss.grad_norm([torch.ones(10)])
    with pytest.raises(ValueError):
        mss.grad_norm([torch.ones(4, 6, device="cuda").t()])
    with pytest.raises(ValueError):
        mss.clip_grads([g], 1.0, out=[])
    with pytest.raises(TypeError):
        mss.clip_grads([g], 1.0, out=[torch.ones(10, device="cuda", dtype=torch.bfloat16)])
    for bad in ([g, g], [g, g[5:]], [g[:6], g[5:]]):
        with pytest.raises(mss.MssError) as err:
            mss.clip_grads(bad, 1.0)
        assert err.value.status == -3
    assert mss.grad_norm([g, g]).item() == pytest.approx(20 ** 0.5)      # a norm may read one twice
    for max_norm, scale in ((-1.0, 1.0), (float("inf"), 1.0), (float("nan"), 1.0), (1.0, 0.0), (1.0, -1.0),
                            (1.0, float("inf"))):
        with pytest.raises(mss.MssError) as err:
            mss.clip_grads([g], max_norm, scale=scale)
        assert err.value.status == -1
    assert (g == 1).all()


def test_a_factor_of_one_changes_no_value():
    """Out of place too, down to the smallest subnormal; and one of a power of two rounds once."""
    g = torch.tensor([1.4e-45, -4.2e-45, 1e-39, -0.0, 1.5, -3e38], device="cuda")
    b = (torch.arange(1, 200).float() * 2.0 ** -133).bfloat16().cuda()
    for grads in ([g], [b], [g, b]):
        same = [torch.empty_like(v) for v in grads]
        mss.clip_grads(grads, 3.4e38, out=same)
        assert all(torch.equal(s.view(torch.uint8), v.view(torch.uint8)) for s, v in zip(same, grads))
    twice, _ = mss.clip_grads([g[:5]], 1e6, scale=2.0, out=[torch.empty(5, device="cuda")])
    assert torch.equal(twice[0].cpu(), g[:5].cpu() * 2)
