"""The float64 forms of the embedding, the head's loss and clipping: closed forms, autograd and
central differences."""
from __future__ import annotations

import math

import pytest
import torch

import ends_ref as ref
from ends_util import generator, normal


def test_embedding_by_hand():
    w = torch.tensor([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    ids = torch.tensor([2, -1, 0, 3, 2])
    y, _ = ref.embedding(ids, w, 0.5, torch.float32)
    assert torch.equal(y, torch.tensor([[2.5, 3], [0, 0], [0.5, 1], [0, 0], [2.5, 3]], dtype=torch.float64))
    dy = torch.tensor([[1.0, 10], [2, 20], [3, 30], [4, 40], [5, 50]])
    dw, _ = ref.embedding_backward(ids, dy, 3, 0.5, torch.float32)
    assert torch.equal(dw, torch.tensor([[1.5, 15], [0, 0], [3, 30]], dtype=torch.float64))
    dw, bound = ref.embedding_backward(ids, dy, 3, 0.5, torch.float32, before=w)
    assert torch.equal(dw, torch.tensor([[2.5, 17], [3, 4], [8, 36]], dtype=torch.float64))
    assert (bound[1] == 0).all()


def test_equal_logits():
    """Rows of zeros: lse = log V, p = 1 / V."""
    x, w = torch.zeros(3, 4), torch.randn(5, 4)
    t = torch.tensor([1, -100, 4])
    g = ref.head(x, w, t, 2.0, torch.ones(3))
    assert torch.allclose(g["lse"][0], torch.full((3,), math.log(5), dtype=torch.float64))
    assert torch.allclose(g["loss"][0], torch.tensor([math.log(5), 0, math.log(5)], dtype=torch.float64))
    want = 2.0 * (w.double().mean(0) - w[1].double())
    assert torch.allclose(g["dx"][0][0], want) and (g["dx"][0][1] == 0).all()
    assert (g["dweight"][0] == 0).all()


@pytest.mark.parametrize("with_lse", [False, True])
def test_head_against_autograd_and_differences(with_lse):
    g = generator(3)
    M, V, D, s = 7, 11, 5, 0.7
    x, w = normal(g, M, D).double(), normal(g, V, D).double()
    t = torch.tensor([0, 10, 3, -1, 3, 11, 7])
    dloss = normal(g, M).double()
    dlse = normal(g, M).double() if with_lse else None
    got = ref.head(x.float(), w.float(), t, s, dloss, dlse)
    x, w = x.float().double().requires_grad_(), w.float().double().requires_grad_()

    def total(x, w):
        logits = s * (x @ w.t())
        inside = (t >= 0) & (t < V)
        lse = torch.logsumexp(logits, 1)
        loss = torch.where(inside, lse - logits.gather(1, t.clamp(0, V - 1)[:, None])[:, 0], 0.0)
        return (dloss * loss).sum() + ((dlse * lse * inside).sum() if with_lse else 0.0)

    total(x, w).backward()
    assert torch.allclose(got["dx"][0], x.grad, atol=1e-12)
    assert torch.allclose(got["dweight"][0], w.grad, atol=1e-12)
    h = 1e-5
    for v, name in ((x, "dx"), (w, "dweight")):
        d = torch.randn(v.shape, dtype=torch.float64, generator=g)
        with torch.no_grad():
            a = (x + h * d, w) if v is x else (x, w + h * d)
            b = (x - h * d, w) if v is x else (x, w - h * d)
            slope = (total(*a) - total(*b)) / (2 * h)
        assert abs(slope - (got[name][0] * d).sum()) < 1e-7


def test_clip_by_hand():
    g = [torch.tensor([3.0, 0.0]), torch.tensor([[4.0]])]
    (norm, _), outs = ref.clip(g, 2.0, 0.5, [torch.float32] * 2)
    assert norm == 2.5 and torch.allclose(outs[0][0], torch.tensor([1.2, 0], dtype=torch.float64))
    (norm, _), outs = ref.clip(g, 5.0, 0.5, [torch.float32] * 2)
    assert torch.equal(outs[1][0], torch.tensor([[2.0]], dtype=torch.float64))
    (norm, _), outs = ref.clip([torch.tensor([float("inf"), 1.0])], 1.0, 0.5, [torch.float32])
    assert norm == float("inf") and outs[0][0][1] == 1
