"""The head's loss and its gradients against float64."""
from __future__ import annotations

import pytest
import torch

import ends_ref as ref
import mamba_selective_scan_causal_amd as mss
from ends_util import TYPES, check, generator, normal, some_ids, spread
from gpu_util import announce

pytestmark = pytest.mark.gpu

# rows, vocabulary, width: below, at and past the tiles' 128 and 256 and their 128 bytes of a row
SIZES = [(1, 1, 1), (1, 300, 64), (5, 2, 8), (8, 4097, 128), (17, 129, 33), (64, 256, 64), (65, 255, 72),
         (128, 128, 136), (129, 1000, 100), (257, 513, 200), (300, 2000, 65), (700, 300, 320)]


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


def case(seed, M, V, D, t, idt=torch.int64, spread_out=3.0):
    """Logits with a standard deviation of about `spread_out` on top of which rows lean to targets."""
    g = generator(seed)
    w = normal(g, V, D, std=D ** -0.5, dtype=t)
    targets = some_ids(g, M, V, idt)
    lean = torch.rand(M, 1, generator=g) * 6
    x = (normal(g, M, D, std=spread_out) + lean * w.float()[targets.clamp(0, V - 1).long()]).to(t)
    return x, w, targets, normal(g, M, std=1.0 / M), normal(g, M, std=0.1 / M)


def run(x, w, targets, dloss, dlse, **kw):
    a = [v.cuda() for v in (x, w, targets)]
    loss, lse = mss.head_loss(*a, **kw)
    grads = mss.head_loss_backward(*a, lse, dloss.cuda(), None if dlse is None else dlse.cuda(), **kw)
    torch.cuda.synchronize()
    return dict(grads, loss=loss, lse=lse)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,V,D", SIZES)
def test_loss_and_gradients(dtype, M, V, D):
    x, w, targets, dloss, dlse = case(M + V + D, M, V, D, TYPES[dtype], torch.int32 if M % 2 else torch.int64)
    dlse = dlse if D % 2 else None
    got = run(x, w, targets, dloss, dlse, logit_scale=0.8)
    want = ref.head(x, w, targets, 0.8, dloss, dlse)
    for k in want:
        announce(f"{k} {check(got[k], want[k], k):.2f} of the bound")


@pytest.mark.parametrize("dtype", TYPES)
def test_several_pieces_of_the_vocabulary(dtype):
    """Sizes whose gradients of the logits do not fit the workspace at once, and whose dx is split."""
    t = TYPES[dtype]
    M, V, D = (40000, 8001, 24) if dtype != "f32" else (40000, 4001, 20)
    need = mss.head_workspace_bytes(mss.OP_HEAD_LOSS_BACKWARD, rows=M, vocab=V, width=D, dtype=t)
    assert need < 2 * M * V * t.itemsize
    x, w, targets, dloss, dlse = [v.cuda() for v in case(1, M, V, D, t)]
    got = run(x, w, targets, dloss, dlse)
    want = ref.head(x, w, targets, 1.0, dloss, dlse)
    for k in want:
        check(got[k], [v.cpu() for v in want[k]], k)


def test_a_long_vocabulary_of_few_rows():
    x, w, targets, dloss, _ = case(2, 9, 70001, 40, torch.bfloat16)
    got = run(x, w, targets, dloss, None)
    want = ref.head(x, w, targets, 1.0, dloss)
    for k in want:
        check(got[k], want[k], k)


def test_large_logits():
    """Logits of some thousands: nothing overflows, a certain row has loss 0 and no gradient."""
    t = torch.float32
    M, V, D = 40, 300, 64
    x, w, targets, dloss, _ = case(3, M, V, D, t, spread_out=1000.0)
    x[5] = 4000.0 * w[targets[5].clamp(0, V - 1)] / w[targets[5].clamp(0, V - 1)].norm()
    got = run(x, w, targets, dloss, None)
    want = ref.head(x, w, targets, 1.0, dloss)
    for k in want:
        check(got[k], want[k], k)


@pytest.mark.parametrize("dtype", TYPES)
def test_padded_rows_take_no_part(dtype):
    """NaN in a padded row's x, dloss and dlse reaches nothing; a batch of padding only has no gradients."""
    t = TYPES[dtype]
    x, w, targets, dloss, dlse = case(4, 150, 200, 48, t)
    off = (targets < 0) | (targets >= 200)
    assert off.any() and not off.all()
    clean = run(x, w, targets, dloss, dlse)
    x[off], dloss[off], dlse[off] = float("nan"), float("nan"), float("inf")
    got = run(x, w, targets, dloss, dlse)
    on = ~off.cuda()
    assert (got["loss"][~on] == 0).all() and (got["dx"][~on] == 0).all()
    for k in ("loss", "lse", "dx"):
        assert torch.equal(got[k][on], clean[k][on])
    assert torch.equal(got["dweight"], clean["dweight"])
    none = run(x, w, torch.full_like(targets, -100), dloss, dlse)
    assert (none["loss"] == 0).all() and (none["dx"] == 0).all() and (none["dweight"] == 0).all()


def test_a_row_of_nan_stays_in_its_row():
    x, w, targets, dloss, _ = case(5, 70, 90, 64, torch.bfloat16)
    targets = targets.clamp(0, 89)
    clean = run(x, w, targets, dloss, None)
    x[3] = float("nan")
    got = run(x, w, targets, dloss, None)
    rest = torch.arange(70, device="cuda") != 3
    assert torch.isnan(got["loss"][3]) and torch.isnan(got["lse"][3]) and torch.isnan(got["dx"][3]).all()
    for k in ("loss", "lse", "dx"):
        assert torch.equal(got[k][rest], clean[k][rest])
    assert torch.isnan(got["dweight"]).all()


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1.0, 65536.0, 1e25])
@pytest.mark.parametrize("dtype", TYPES)
def test_gradients_of_any_size(dtype, size):
    """dloss scaled by a power of two, as a mean over many rows or a loss scale brings it: the
    gradients keep their digits (they are compared before the scale would round them away)."""
    t = TYPES[dtype]
    x, w, targets, dloss, dlse = case(6, 100, 500, 64, t)
    base = run(x, w, targets, dloss, dlse)
    scale = 2.0 ** round(torch.log2(torch.tensor(size)).item())
    got = run(x, w, targets, dloss * scale, dlse * scale)
    fits = torch.finfo(t)
    for k in ("dx", "dweight"):
        want = base[k].double() * scale
        # the same digits where neither side is a subnormal or overflows
        clear = (want.abs() >= 4 * fits.tiny) & (want.abs() <= fits.max / 2) & (base[k].abs() >= 4 * fits.tiny)
        assert torch.allclose(got[k].double()[clear], want[clear], rtol=2 * ref.HALF[t], atol=0), (k, dtype, size)


def test_no_gradient_at_all():
    x, w, targets, dloss, _ = case(7, 40, 60, 32, torch.float16)
    got = run(x, w, targets, torch.zeros_like(dloss), None)
    assert (got["dx"] == 0).all() and (got["dweight"] == 0).all()


@pytest.mark.parametrize("dtype,D", [("bf16", 72), ("f32", 36), ("bf16", 71), ("f32", 33), ("f16", 129)])
def test_strided_rows_and_what_lies_around(dtype, D):
    t = TYPES[dtype]
    M, V = 140, 270
    x, w, targets, dloss, dlse = [v.cuda() for v in case(8, M, V, D, t)]
    want = run(x, w, targets, dloss, dlse)
    xs, _ = spread(x)
    ws, _ = spread(w)
    dxs, dxw = spread(torch.zeros_like(x))
    dws, dww = spread(torch.zeros_like(w))
    loss = torch.full((M + 2,), 7.0, device="cuda")
    lse = torch.full((M + 2,), 7.0, device="cuda")
    mss.head_loss(xs, ws, targets, out=(loss[1:-1], lse[1:-1]))
    mss.head_loss_backward(xs, ws, targets, lse[1:-1], dloss, dlse, out=dict(dx=dxs, dweight=dws))
    torch.cuda.synchronize()
    for got, k in ((loss[1:-1], "loss"), (lse[1:-1], "lse"), (dxs, "dx"), (dws, "dweight")):
        assert torch.equal(got, want[k]), k
    assert (loss[[0, -1]] == 7).all() and (lse[[0, -1]] == 7).all()
    for wide in (dxw, dww):
        assert torch.isnan(wide[:, :1]).all() and torch.isnan(wide[:, D + 1:]).all()


def test_one_gradient_alone():
    x, w, targets, dloss, dlse = [v.cuda() for v in case(9, 200, 700, 96, torch.bfloat16)]
    _, lse = mss.head_loss(x, w, targets)
    both = mss.head_loss_backward(x, w, targets, lse, dloss, dlse)
    a = mss.head_loss_backward(x, w, targets, lse, dloss, dlse, need_dweight=False)
    b = mss.head_loss_backward(x, w, targets, lse, dloss, dlse, need_dx=False)
    assert a["dweight"] is None and torch.equal(a["dx"], both["dx"])
    assert b["dx"] is None and torch.equal(b["dweight"], both["dweight"])
    assert mss.head_loss_backward(x, w, targets, lse, dloss, need_dx=False, need_dweight=False) == dict(
        dx=None, dweight=None)


def test_no_rows():
    w = torch.ones(30, 16, device="cuda")
    x, t, f = torch.empty(0, 16, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    loss, lse = mss.head_loss(x, w, t)
    assert loss.shape == lse.shape == (0,)
    g = mss.head_loss_backward(x, w, t, f, f, out=dict(dweight=torch.ones(30, 16, device="cuda")))
    assert (g["dweight"] == 0).all() and g["dx"].shape == (0, 16)


def test_gradients_against_differences_of_the_kernels():
    """fp32, along a direction: (loss(x + h d) - loss(x - h d)) / 2h against <dx, d>.  The losses are
    off by the reference's bounds; the difference by h^2 / 6 times the third derivative, a third
    cumulant of the logits' slopes, which is at most their range cubed."""
    M, V, D, h = 60, 150, 64, 0.05
    x, w, targets, _, _ = case(10, M, V, D, torch.float32, spread_out=1.0)
    targets = targets.clamp(0, V - 1)
    got = run(x, w, targets, torch.ones(M), None)
    want = ref.head(x, w, targets, 1.0, torch.ones(M))
    g = generator(11)
    d, e = normal(g, M, D, std=D ** -0.5), normal(g, V, D, std=0.1 * D ** -0.5)

    def slopes(x1, w1, x0, w0, along):
        sides = [mss.head_loss(a.cuda(), b.cuda(), targets.cuda())[0].double().cpu() for a, b in ((x1, w1), (x0, w0))]
        off = sum(ref.head(a, b, targets, 1.0)["loss"][1] for a, b in ((x1, w1), (x0, w0))) / (2 * h)
        reach = along.max(1).values - along.min(1).values
        return (sides[0] - sides[1]) / (2 * h), off + h * h / 6 * (1.1 * reach) ** 3

    slope, off = slopes(x + h * d, w, x - h * d, w, d.double() @ w.double().t())
    announce(f"slopes of {slope.abs().mean():.2g} within {off.max():.2g}")
    assert off.max() < 0.02 * slope.abs().max()
    exact = (got["dx"].double().cpu() * d.double()).sum(1)
    assert ((slope - exact).abs() <= off + (want["dx"][1] * d.abs().double()).sum(1)).all()
    slope, off = slopes(x, w + h * e, x, w - h * e, x.double() @ e.double().t())
    exact = (got["dweight"].double().cpu() * e.double()).sum()
    assert abs(slope.sum() - exact) <= off.sum() + (want["dweight"][1] * e.abs().double()).sum()


def test_same_bits_every_time():
    x, w, targets, dloss, dlse = [v.cuda() for v in case(12, 1000, 3000, 128, torch.bfloat16)]
    first = run(x, w, targets, dloss, dlse)
    for _ in range(4):
        again = run(x, w, targets, dloss, dlse)
        assert all(torch.equal(first[k], again[k]) for k in first)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,V,D", [(66000, 40, 48), (70001, 257, 33), (2500, 100, 520), (20000, 256, 64)])
def test_many_rows_of_a_small_vocabulary(dtype, M, V, D):
    """dweight is a few tiles with a long sum over the rows, which is split; the gradients' largest
    factor is that of one of the last rows."""
    t = TYPES[dtype]
    x, w, targets, dloss, dlse = case(13, M, V, D, t)
    targets[-2], dloss[-2] = 1, 64.0 / M
    x, w, targets, dloss, dlse = [v.cuda() for v in (x, w, targets, dloss, dlse)]
    got = run(x, w, targets, dloss, dlse)
    want = ref.head(x, w, targets, 1.0, dloss, dlse)
    for k in want:
        announce(f"{k} {check(got[k], [v.cpu() for v in want[k]], k):.2f} of the bound")
    alone = mss.head_loss_backward(x, w, targets, got["lse"], dloss, dlse, need_dx=False)
    assert torch.equal(alone["dweight"], got["dweight"])


@pytest.mark.parametrize("dtype,M,V,D", [
    ("bf16", 31, 600, 64), ("f16", 32, 1000, 40), ("bf16", 33, 1000, 64), ("f32", 32, 500, 36), ("f32", 255, 300, 64),
    ("f32", 256, 300, 64), ("f32", 257, 300, 63), ("f16", 1023, 520, 72), ("bf16", 1024, 520, 72), ("bf16", 1023, 333, 71),
    ("f16", 1024, 333, 71), ("bf16", 1025, 261, 129), ("f32", 1024, 261, 33), ("f32", 1030, 200, 70)])
def test_where_the_row_counts_change_the_way(dtype, M, V, D):
    """Around 32, 256 and 1024 rows, dense and in strides that put rows at any element: the same bits."""
    t = TYPES[dtype]
    x, w, targets, dloss, dlse = [v.cuda() for v in case(14, M, V, D, t)]
    got = run(x, w, targets, dloss, dlse)
    want = ref.head(x, w, targets, 1.0, dloss, dlse)
    for k in want:
        announce(f"{k} {check(got[k], [v.cpu() for v in want[k]], k):.2f} of the bound")
    again = run(spread(x)[0], spread(w)[0], targets, dloss, dlse)
    for k in want:
        assert torch.equal(got[k], again[k]), k


@pytest.mark.parametrize("scale", [-1.5, 0.0])
@pytest.mark.parametrize("dtype", TYPES)
def test_logit_scales_of_any_sign(dtype, scale):
    x, w, targets, dloss, dlse = case(15, 90, 310, 56, TYPES[dtype])
    got = run(x, w, targets, dloss, dlse, logit_scale=scale)
    want = ref.head(x, w, targets, scale, dloss, dlse)
    for k in want:
        check(got[k], want[k], k)


def test_a_vocabulary_in_pieces_of_the_forward():
    x, w, targets, dloss, dlse = [v.cuda() for v in case(16, 37, 270001, 24, torch.bfloat16)]
    got = run(x, w, targets, dloss, dlse)
    want = ref.head(x, w, targets, 1.0, dloss, dlse)
    for k in want:
        check(got[k], [v.cpu() for v in want[k]], k)


@pytest.mark.parametrize("M", [30484, 33001])
def test_rows_in_pieces_of_the_forward(M):
    """More partial sums than are held at a time; the last piece has a few rows, or thousands."""
    V = 70001
    x, w, targets, _, _ = [v.cuda() for v in case(17, M, V, 8, torch.bfloat16)]
    need = mss.head_workspace_bytes(mss.OP_HEAD_LOSS, rows=M, vocab=V, width=8, dtype=torch.bfloat16)
    assert need < (V // 64 + 2) * M * 8 + 4 * M        # of all rows at once
    loss, lse = mss.head_loss(x, w, targets)
    rows = torch.cat([torch.arange(40), torch.arange(30400, 30484), torch.arange(M - 40, M)])
    want = ref.head(x[rows], w, targets[rows], 1.0)
    check(loss[rows], [v.cpu() for v in want["loss"]], "loss")
    check(lse[rows], [v.cpu() for v in want["lse"]], "lse")
    # and the rest by their own sums in fp32, in which a logit and its exponential are off by little
    for r in range(0, M, 4000):
        l = x[r:r + 4000].float() @ w.float().t()
        assert torch.allclose(lse[r:r + 4000], torch.logsumexp(l, 1), rtol=1e-5, atol=1e-5)


def test_more_rows_than_a_gibibyte_of_gradients():
    M, V, D = 90000, 4900, 16
    x, w, targets, dloss, dlse = [v.cuda() for v in case(18, M, V, D, torch.float16)]
    need = mss.head_workspace_bytes(mss.OP_HEAD_LOSS_BACKWARD, rows=M, vocab=V, width=D, dtype=torch.float16)
    assert 2 ** 30 < need < 2 * 2 * M * V            # dl and its transpose, a piece of the vocabulary at a time
    got = run(x, w, targets, dloss, dlse)
    want = ref.head(x, w, targets, 1.0, dloss, dlse)
    for k in want:
        check(got[k], [v.cpu() for v in want[k]], k)
