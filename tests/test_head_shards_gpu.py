"""The head over a vocabulary in shards: loss, log sum and both gradients are the whole vocabulary's."""
from __future__ import annotations

import pytest
import torch

import ends_ref as ref
import mamba_selective_scan_causal_amd as mss
from ends_util import TYPES, check
from gpu_util import announce
from test_head_gpu import case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


def sharded(x, w, targets, dloss, dlse, ends):
    """What each shard's program does, with the sums over the shards in between."""
    V = w.shape[0]
    valid = (targets >= 0) & (targets < V)
    parts = [(a, w[a:b]) for a, b in zip(ends, ends[1:])]
    here = [valid & (targets >= a) & (targets < a + len(v)) for a, v in parts]
    local = [torch.where(h, targets - a, -100) for (a, v), h in zip(parts, here)]
    each = [mss.head_loss(x, v, t) for (a, v), t in zip(parts, local)]
    lse = torch.logsumexp(torch.stack([s for _, s in each]), 0)
    own = sum(torch.where(h, s - l, 0.0) for (l, s), h in zip(each, here))
    loss = torch.where(valid, lse - own, 0.0)
    grads = []
    for (a, v), t, h in zip(parts, local, here):
        away = valid & ~h
        up = torch.where(away, 0.0, dloss)
        more = torch.where(away, dloss + dlse, dlse)
        grads.append(mss.head_loss_backward(x, v, torch.where(away, 0, t), lse, up, more))
    return loss, lse, [g["dx"] for g in grads], torch.cat([g["dweight"] for g in grads])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,V,D,ends", [(200, 500, 64, (0, 250, 500)), (33, 1001, 40, (0, 1, 700, 1001)),
                                        (1300, 640, 65, (0, 320, 640))])
def test_gradients_over_shards(dtype, M, V, D, ends):
    t = TYPES[dtype]
    x, w, targets, dloss, dlse = case(M, M, V, D, t)
    loss, lse, dxs, dw = sharded(*[v.cuda() for v in (x, w, targets, dloss, dlse)], ends)
    want = ref.head(x, w, targets, 1.0, dloss, dlse)
    # joined in fp32: exponentials and a sum of a few, a log, two differences
    more = 8 * ref.U * (1 + want["lse"][0].abs())
    for k, got in (("lse", lse), ("loss", loss)):
        check(got, (want[k][0], want[k][1] + more), k)
    # so p is off by that, and each shard's dx is rounded once: by half a step of its value, or half the
    # least step where it is a subnormal (fp16: 2^-25 for each shard, which 'rounded' counts once)
    p = torch.softmax(x.double() @ w.double().t(), 1)
    p *= (more * (dloss.abs() + dlse.abs()) * ((targets >= 0) & (targets < V))).double()[:, None]
    dx = sum(g.double().cpu() for g in dxs)
    rounds = sum(ref.HALF[t] * g.double().abs().cpu() + ref.TINY[t] for g in dxs)
    check(dx, (want["dx"][0], want["dx"][1] + p @ w.double().abs() + rounds), "dx")
    value, bound = want["dweight"]
    check(dw, (value, bound + p.t() @ x.double().abs() * (1 + ref.HALF[t])), "dweight")
    padded = ((targets < 0) | (targets >= V)).cuda()
    assert all((g[padded] == 0).all() for g in dxs)
