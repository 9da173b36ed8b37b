"""Clipping of lists with more chunks than workgroups, in each size of chunk, and the embedding at widths
that take several workgroups or several rounds of a wave for a row."""
from __future__ import annotations

import pytest
import torch

import ends_ref as ref
import mamba_selective_scan_causal_amd as mss
from ends_util import TYPES, check, generator, normal, some_ids, spread
from gpu_util import announce
from test_embed_gpu import PAIRS

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


# elements in all: chunks of 2048 up to 16.8 million, then 4096, 8192 and 16384; the short tensors between
# two long ones (with 40 the list goes in two parts of 96 tensors at most, each with its own chunks)
TOTALS = {"2048": (16_000_003, 20), "4096": (21_000_007, 20), "8192": (45_000_011, 20), "16384": (80_000_023, 20),
          "4096 and 4096": (46_000_003, 40)}


def many(total, short, types):
    """Long tensors with short ones between them, whose ends fall anywhere in a chunk."""
    g = torch.Generator(device="cuda").manual_seed(total)
    sizes = []
    for k in range(4):
        sizes += [total // 4 - 977 * k - 1000 * (k == 0)] + [(37 * j * j + k) % 5001 + 1 for j in range(short)]
    return [torch.randn(n, generator=g, device="cuda").mul_(10.0 ** -(k % 3)).to(TYPES[types[k % len(types)]])
            for k, n in enumerate(sizes)]


def compare(got, want, what):
    value, bound = want
    assert got.shape == value.shape and ((got.double() - value).abs() <= bound).all(), what


@pytest.mark.parametrize("where", ["in place", "same types", "f32", "mixed"])
@pytest.mark.parametrize("chunk", TOTALS)
def test_more_chunks_than_workgroups(chunk, where):
    grads = many(*TOTALS[chunk], ["bf16", "f32", "f16"] if where != "f32" else ["bf16", "f16"])
    assert sum(g.numel() for g in grads) / int(chunk.split()[0]) > 2048
    kept = [g.clone() for g in grads]
    types = [torch.float32 if where == "f32" else g.dtype for g in grads]
    (norm, off), outs = ref.clip(kept, 1.0, 0.5, types)
    to = None if where == "in place" else [
        g if where == "mixed" and k % 2 else torch.full(g.shape, 7.0, dtype=t, device="cuda")
        for k, (g, t) in enumerate(zip(grads, types))]
    n0 = mss.grad_norm(grads, scale=0.5)
    # a factor of one: in place it is not even read, elsewhere copied
    same, n1 = mss.clip_grads(grads, 1e9, scale=1.0, out=to)
    assert all(torch.equal(a, b) for a, b in zip(same, kept)) and torch.equal(2 * n0, n1)
    got, n = mss.clip_grads(grads, 1.0, scale=0.5, out=to)
    assert torch.equal(n, n0) and abs(n.item() - norm) <= off
    for k, (o, want) in enumerate(zip(got, outs)):
        compare(o, want, f"tensor {k}")
        if to is not None and to[k] is not grads[k]:
            assert torch.equal(grads[k], kept[k])


@pytest.mark.parametrize("table,rows", PAIRS)
@pytest.mark.parametrize("D", [1025, 2049, 2561, 4100, 4097])
def test_wide_rows(table, rows, D):
    M, V = 700, 90
    g = generator(D)
    tw, ty = TYPES[table], TYPES[rows]
    ids, w, dy = some_ids(g, M, V), normal(g, V, D, dtype=tw), normal(g, M, D, dtype=ty)
    ids[100:105], w[7] = 7, 0
    more = normal(g, V, D, dtype=tw)
    i, wc, dyc = ids.cuda(), w.cuda(), dy.cuda()
    y = mss.embedding(i, wc, scale=1.7, out_dtype=ty)
    dw = mss.embedding_backward(i, dyc, vocab=V, scale=-0.6, dtype=tw)
    acc = mss.embedding_backward(i, dyc, vocab=V, scale=-0.6, accumulate=True, out=more.cuda())
    check(y, ref.embedding(ids, w, 1.7, ty), "y")
    check(dw, ref.embedding_backward(ids, dy, V, -0.6, tw), "dweight")
    check(acc, ref.embedding_backward(ids, dy, V, -0.6, tw, before=more), "accumulated")
    ys, wide = spread(torch.zeros(M, D, dtype=ty, device="cuda"))
    mss.embedding(i, spread(wc)[0], scale=1.7, out=ys)
    dws, dwide = spread(torch.ones(V, D, dtype=tw, device="cuda"))
    mss.embedding_backward(i, spread(dyc)[0], vocab=V, scale=-0.6, out=dws)
    accs, awide = spread(more.cuda())
    mss.embedding_backward(i, spread(dyc)[0], vocab=V, scale=-0.6, out=accs, accumulate=True)
    for a, b, around in ((ys, y, wide), (dws, dw, dwide), (accs, acc, awide)):
        assert torch.equal(a, b) and torch.isnan(around[:, :1]).all() and torch.isnan(around[:, D + 1:]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_token_in_many_runs_of_wide_rows(dtype):
    """Its parts are added up by whole workgroups, for each group of columns."""
    M, V, D, t = 6000, 5, 2561, TYPES[dtype]
    g = generator(3)
    ids, dy = torch.randint(0, V, (M,), generator=g), normal(g, M, D, dtype=t)
    dw = mss.embedding_backward(ids.cuda(), dy.cuda(), vocab=V, dtype=torch.float32)
    check(dw, ref.embedding_backward(ids, dy, V, 1.0, torch.float32), "dweight")
