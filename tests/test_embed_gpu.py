"""The embedding and its gradient against float64."""
from __future__ import annotations

import pytest
import torch

import ends_ref as ref
import mamba_selective_scan_causal_amd as mss
from ends_util import TYPES, check, generator, normal, some_ids, spread
from gpu_util import announce

pytestmark = pytest.mark.gpu

PAIRS = [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32"), ("f16", "f32"), ("f32", "bf16"),
         ("f32", "f16")]
# rows, vocabulary, width: one of each; below, at and past a wave, a sort tile, a run of positions
SIZES = [(1, 1, 1), (3, 2, 7), (31, 5, 64), (32, 40, 65), (33, 7, 512), (64, 1000, 8), (100, 3, 129), (257, 2000, 1001),
         (2048, 33, 72), (2049, 1024, 40), (5000, 70000, 16), (4097, 1023, 200)]


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


@pytest.mark.parametrize("table,rows", PAIRS)
@pytest.mark.parametrize("M,V,D", SIZES)
def test_lookup_and_gradient(table, rows, M, V, D):
    g = generator(M + V + D)
    tw, ty = TYPES[table], TYPES[rows]
    idt = torch.int32 if (M + D) % 2 else torch.int64
    ids, w, dy = some_ids(g, M, V, idt), normal(g, V, D, dtype=tw), normal(g, M, D, dtype=ty)
    y = mss.embedding(ids.cuda(), w.cuda(), scale=1.7, out_dtype=ty)
    dw = mss.embedding_backward(ids.cuda(), dy.cuda(), vocab=V, scale=-0.6, dtype=tw)
    more = normal(g, V, D, dtype=tw)
    acc = mss.embedding_backward(ids.cuda(), dy.cuda(), vocab=V, scale=-0.6, accumulate=True, out=more.cuda())
    torch.cuda.synchronize()
    assert y.dtype == ty and dw.dtype == tw
    check(y, ref.embedding(ids, w, 1.7, ty), "y")
    check(dw, ref.embedding_backward(ids, dy, V, -0.6, tw), "dweight")
    check(acc, ref.embedding_backward(ids, dy, V, -0.6, tw, before=more), "accumulated")


@pytest.mark.parametrize("M,V", [(1000, 1), (9000, 3), (33, 1), (70, 2)])
def test_few_tokens_in_many_places(M, V):
    """Tokens that reach over many runs of positions, from one place to all of them."""
    g = generator(M)
    ids = torch.randint(0, V, (M,), generator=g)
    dy = normal(g, M, 24, dtype=torch.bfloat16)
    dw = mss.embedding_backward(ids.cuda(), dy.cuda(), vocab=V, dtype=torch.float32)
    check(dw, ref.embedding_backward(ids, dy, V, 1.0, torch.float32), "dweight")


@pytest.mark.parametrize("M,V", [(3000, 2 ** 21 + 5), (40000, 2 ** 21 + 5), (40000, 3), (150000, 1000), (32768, 70000),
                                 (32767, 511), (32769, 512), (1025, 2 ** 25)])
def test_more_digits_and_larger_tiles(M, V):
    """Ids of three digits; more positions than fit the smallest tiles of the sort."""
    g = generator(M)
    ids, dy = some_ids(g, M, V), normal(g, M, 4 if V < 2 ** 22 else 1)
    dw = mss.embedding_backward(ids.cuda(), dy.cuda(), vocab=V)
    check(dw, ref.embedding_backward(ids, dy, V, 1.0, torch.float32), "dweight")


def test_all_padding_and_none():
    g = generator(1)
    dy = normal(g, 50, 40)
    for ids in (torch.full((50,), -1), torch.full((50,), 9), torch.full((50,), 2 ** 40), torch.full((50,), -2 ** 62)):
        out = torch.full((9, 40), 7.0, device="cuda")
        dw = mss.embedding_backward(ids.cuda(), dy.cuda(), vocab=9, out=out)
        assert (dw == 0).all()
        out.fill_(7)
        mss.embedding_backward(ids.cuda(), dy.cuda(), vocab=9, out=out, accumulate=True)
        assert (out == 7).all()
        y = mss.embedding(ids.cuda(), torch.full((9, 40), float("nan"), device="cuda"))
        assert (y == 0).all()


def test_no_rows_no_vocabulary():
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert mss.embedding(none, torch.ones(4, 8, device="cuda")).shape == (0, 8)
    dw = mss.embedding_backward(none, torch.empty(0, 8, device="cuda"), vocab=40, out=torch.ones(40, 8, device="cuda"))
    assert (dw == 0).all()
    kept = mss.embedding_backward(none, torch.empty(0, 8, device="cuda"), vocab=4, accumulate=True,
                                  out=torch.ones(4, 8, device="cuda"))
    assert (kept == 1).all()
    ids = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert (mss.embedding(ids, torch.empty(0, 8, device="cuda")) == 0).all()
    assert mss.embedding_backward(ids, torch.ones(3, 8, device="cuda"), vocab=0).shape == (0, 8)


def test_padded_gradients_are_not_read():
    """NaN in the rows of padded places stays out of the sums; NaN of a token stays in its row."""
    ids = torch.tensor([1, -1, 3, 1, 8, 3] * 20)
    dy = torch.ones(120, 10)
    dy[(ids < 0) | (ids >= 8)] = float("nan")
    dy[2] = float("inf")
    dw = mss.embedding_backward(ids.cuda(), dy.cuda(), vocab=8).cpu()
    assert (dw[1] == 40).all() and torch.isinf(dw[3]).all() and (dw[[0, 2, 4, 5, 6, 7]] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_strided_rows_and_what_lies_around(dtype):
    """Columns of wider buffers, off every wider alignment: the same bits, and nothing else written."""
    g = generator(5)
    t = TYPES[dtype]
    M, V, D = 300, 90, 131
    ids, w, dy = some_ids(g, M, V).cuda(), normal(g, V, D, dtype=t).cuda(), normal(g, M, D, dtype=t).cuda()
    y, dw = mss.embedding(ids, w), mss.embedding_backward(ids, dy, vocab=V)
    ws, _ = spread(w)
    dys, _ = spread(dy)
    outs, out = spread(torch.zeros_like(dy))
    assert torch.equal(mss.embedding(ids, ws, out=outs), y)
    dws, dwide = spread(torch.ones_like(w))
    assert torch.equal(mss.embedding_backward(ids, dys, vocab=V, out=dws), dw)
    base = normal(g, V, D, dtype=t).cuda()
    accs, awide = spread(base.clone())
    mss.embedding_backward(ids, dys, vocab=V, out=accs, accumulate=True)
    assert torch.equal(accs, mss.embedding_backward(ids, dy, vocab=V, out=base.clone(), accumulate=True))
    for wide in (out, dwide, awide):
        assert torch.isnan(wide[:, :1]).all() and torch.isnan(wide[:, D + 1:]).all()


def test_same_bits_every_time():
    g = generator(6)
    ids, dy = some_ids(g, 20000, 500).cuda(), normal(g, 20000, 96).cuda()
    first = mss.embedding_backward(ids, dy, vocab=500)
    for _ in range(5):
        assert torch.equal(mss.embedding_backward(ids, dy, vocab=500), first)


def test_the_gradient_of_the_lookup():
    """<dy, y(W + D) - y(W)> = <dW, D>: the lookup is linear."""
    g = generator(7)
    ids, w, d, dy = some_ids(g, 700, 300), normal(g, 300, 48), normal(g, 300, 48), normal(g, 700, 48)
    y = mss.embedding(ids.cuda(), d.cuda(), scale=0.3).double().cpu()
    dw = mss.embedding_backward(ids.cuda(), dy.cuda(), vocab=300, scale=0.3).double().cpu()
    left, right = (dy.double() * y).sum(), (dw * d.double()).sum()
    # 700 x 48 products, each off by at most (n + 4) U with n < 400 places of a token
    assert abs(left - right) <= 404 * ref.U * (dy.double() * y).abs().sum()


def test_as_many_positions_as_there_may_be():
    """2^26 - 1 of them, in rows of one value: sums of ones, exact in fp32."""
    M, V = 2 ** 26 - 1, 5
    ids = (torch.arange(M, dtype=torch.int32, device="cuda") * 7 % 11)
    w = torch.arange(1, V + 1, device="cuda").float().view(V, 1).half()
    y = mss.embedding(ids, w)
    assert torch.equal(y[:, 0], torch.where(ids < V, ids + 1, 0).half())
    dw = mss.embedding_backward(ids, torch.ones(M, 1, device="cuda"), vocab=V)
    want = torch.tensor([float((ids == v).sum()) for v in range(V)], device="cuda")
    assert torch.equal(dw[:, 0], want)
