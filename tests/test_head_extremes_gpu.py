"""The head's loss and gradients where logits are masked, far from zero or infinite."""
from __future__ import annotations

import pytest
import torch

import ends_ref as ref
from ends_util import TYPES, check, generator, normal, spread
from gpu_util import announce
from test_head_gpu import run

pytestmark = pytest.mark.gpu

INF = float("inf")
# what a constant feature times the mask's weight makes of a logit
MASKS = {"bf16": [-1e10, -1e30, -2.5e38, torch.finfo(torch.bfloat16).min, -INF],
         "f32": [-1e10, -1e30, -2.5e38, torch.finfo(torch.float32).min],
         "f16": [-300.0, -65504.0, -INF]}
FEATURE = {"bf16": 1.0, "f32": 1.0, "f16": 60000.0}
# 640 is a multiple of 32, 64, 80, 128 and 160, the columns of one wave
LAYOUTS = {"a middle part": (1000, lambda v: (v >= 300) & (v < 700)), "the last token": (641, lambda v: v == 640),
           "all but one token": (500, lambda v: v != 5), "the first part": (700, lambda v: v < 330)}


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


def masked(seed, M, V, D, dtype, off, value):
    """Feature 0 is a constant, and the weight's column 0 the mask."""
    g, t = generator(seed), TYPES[dtype]
    keep = torch.nonzero(~off)[:, 0]
    w = normal(g, V, D, std=D ** -0.5)
    w[:, 0] = torch.where(off, value, 0.0)
    targets = keep[torch.randint(0, len(keep), (M,), generator=g)]
    x = normal(g, M, D, std=3.0)
    x[:, 0] = FEATURE[dtype]
    return x.to(t), w.to(t), keep, targets, normal(g, M, std=0.1 / M)


def check_masked(x, w, keep, targets, dloss, got, columns):
    """Against the loss over the tokens that are not masked: the others add exp(-large) = 0 to every sum."""
    where = torch.full((w.shape[0],), -100)
    where[keep] = torch.arange(len(keep))
    inside = (targets >= 0) & (targets < w.shape[0])
    want = ref.head(x, w[keep], torch.where(inside, where[targets.clamp(0, w.shape[0] - 1)], -100), 1.0, dloss)
    check(got["loss"], want["loss"], "loss")
    check(got["lse"], want["lse"], "lse")
    check(got["dx"][:, columns], [v[:, columns] for v in want["dx"]], "dx")
    check(got["dweight"][keep.cuda()], want["dweight"], "dweight")
    hidden = torch.ones(w.shape[0], dtype=torch.bool, device="cuda")
    hidden[keep] = False
    assert (got["dweight"][hidden] == 0).all()


@pytest.mark.parametrize("dtype,value", [(t, v) for t in TYPES for v in MASKS[t]])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("M", [5, 40, 300])
def test_masked_tokens(M, layout, dtype, value):
    V, off = LAYOUTS[layout]
    x, w, keep, targets, dloss = masked(M + V, M, V, 72, dtype, off(torch.arange(V)), value)
    got = run(x, w, targets, dloss, None)
    # 0 * -inf is NaN in the gradient of the constant feature
    check_masked(x, w, keep, targets, dloss, got, slice(1 if value == -INF else 0, None))


@pytest.mark.parametrize("scale", [1.0, 0.75, -1.0])
@pytest.mark.parametrize("dtype,a,b", [("bf16", 30, 0), ("bf16", 60, 0), ("bf16", 110, 0), ("f32", 30, 0), ("f32", 60, 0),
                                       ("f32", 110, 0), ("f16", 12, 12)])
def test_logits_far_from_zero(dtype, a, b, scale):
    """Small integers times 2^a and 2^b: exact logits, so far apart that only the largest counts.  lse is that one
    and the loss a difference, both exact; dl is dloss at the largest and -dloss at the target, rounded once."""
    M, V, D, t = 150, 900, 16, TYPES[dtype]
    g = generator(a)
    x = torch.randint(-4, 5, (M, D), generator=g).double()
    w = torch.randint(-4, 5, (V, D), generator=g).double()
    targets = torch.randint(0, V, (M,), generator=g)
    logits = scale * (x @ w.t())
    top, at = logits.max(1)
    alone = (logits == top[:, None]).sum(1) == 1
    assert alone.sum() > M // 4
    dloss = torch.where(alone, normal(g, M, std=1.0 / M), 0.0)
    x, w = x * 2.0 ** a, w * 2.0 ** b
    got = run(x.to(t), w.to(t), targets, dloss, None, logit_scale=scale)
    size = 2.0 ** (a + b)
    assert torch.equal(got["lse"].double().cpu(), top * size)
    assert torch.equal(got["loss"].double().cpu(), (top - logits.gather(1, targets[:, None])[:, 0]) * size)
    dl = torch.zeros(M, V, dtype=torch.float64)
    dl[torch.arange(M), at] += dloss.double()
    dl[torch.arange(M), targets] -= dloss.double()
    for name, left, right, n in (("dx", dl, w, V), ("dweight", dl.t(), x, M)):
        size = abs(scale) * (left.abs() @ right.abs())
        value = scale * (left @ right)
        check(got[name], (value, ref.rounded(value, (ref.HALF[t] + (n + 28) * ref.U) * size, t)), name)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logits_whose_log2_is_beyond_fp32(dtype):
    """2.5e38 log2(e) is not an fp32 number, 2.5e38 is: all logits of a row are it, up to what ordinary
    features change, which is lost in its last place."""
    M, V, D, t = 70, 700, 40, TYPES[dtype]
    x, w, _, targets, dloss = masked(1, M, V, D, dtype, torch.ones(V, dtype=torch.bool) & (torch.arange(V) > 0), 0.0)
    w[:, 0] = 2.5e38
    got = run(x, w, targets, dloss, None)
    most = w[0, 0].double()
    assert ((got["lse"].double().cpu() - most).abs() <= 4 * ref.U * most).all()
    assert (got["loss"].abs().double().cpu() <= 8 * ref.U * most).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_infinite_logits(dtype):
    """lse is inf where a logit is, and so is another target's loss; it is -inf where every logit is."""
    M, V, D = 40, 700, 40
    every = torch.ones(V, dtype=torch.bool)
    x, w, _, targets, dloss = masked(2, M, V, D, dtype, every & (torch.arange(V) < 690), 0.0)
    w[650, 0] = INF
    got = run(x, w, targets, dloss, None)
    assert (got["lse"] == INF).all() and (got["loss"] == INF).all()
    w[:, 0] = -INF
    got = run(x, w, targets, dloss, None)
    assert (got["lse"] == -INF).all()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("D", [72, 33])
@pytest.mark.parametrize("M", [5, 40, 300])
def test_tokens_masked_by_an_infinity_in_fp32(M, D, layout):
    """Operands of the products are three parts each, which an infinity has not."""
    V, off = LAYOUTS[layout]
    x, w, keep, targets, dloss = masked(M + V, M, V, D, "f32", off(torch.arange(V)), -INF)
    got = run(x, w, targets, dloss, None)
    check_masked(x, w, keep, targets, dloss, got, slice(1, None))
    got = run(spread(x)[0], spread(w)[0], targets, dloss, None)
    check_masked(x, w, keep, targets, dloss, got, slice(1, None))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,D", [(5, 72), (40, 33), (300, 64), (1500, 31)])
def test_infinities_here_and_there(dtype, M, D):
    """Infinities of either sign and NaN as the sums of products have them, and in no other row."""
    V, t = 700, TYPES[dtype]
    g = generator(M)
    x, w = normal(g, M, D, std=2.0), normal(g, V, D, std=D ** -0.5)
    targets, dloss = torch.randint(20, V, (M,), generator=g), normal(g, M, std=0.1 / M)
    x, w = x.to(t), w.to(t)
    w[11, 3] = w[12, 3] = INF
    x[1, 3] = 0.0
    x[2, 7] = INF
    x[3, 5] = float("nan")
    x[4, 3] = -1.0
    got = run(x, w, targets, dloss, None)
    logits = torch.stack([(r * w.double()).sum(1) for r in x.double()])
    lse = torch.logsumexp(logits, 1)
    far = logits.max(1).values == INF
    lse[far & ~logits.isnan().any(1)] = INF
    here = got["lse"].double().cpu()
    assert here[1].isnan() and here[3].isnan() and torch.equal(here.isnan(), logits.isnan().any(1))
    assert torch.equal(here == INF, lse == INF) and ((lse == INF).any() or M == 5)
    rest = torch.isfinite(lse)
    assert rest[4]
    keep = torch.tensor([v for v in range(V) if v not in (11, 12)])
    want = ref.head(x[rest], w[keep], torch.where(targets > 12, targets - 2, targets)[rest], 1.0, dloss[rest])
    for k in ("loss", "lse"):
        check(got[k][rest.cuda()], want[k], k)
    columns = [d for d in range(D) if d != 3]
    value, bound = want["dx"]
    check(got["dx"][rest.cuda()][:, columns], (value[:, columns], bound[:, columns]), "dx")
    # a row that has none of it keeps its bits
    w[11:13, 3] = 0.0
    x[1, 3] = 1.0
    a = run(x, w, targets, dloss, None)
    x[2, 7] = x[3, 5] = 1.0
    b = run(x, w, targets, dloss, None)
    same = torch.ones(M, dtype=torch.bool, device="cuda")
    same[2:4] = False
    for k in ("loss", "lse", "dx"):
        assert torch.equal(a[k][same], b[k][same]), k


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,V,D", [(40, 700, 72), (300, 5000, 33), (5, 20000, 64), (1100, 900, 40), (9000, 130, 24)])
def test_padded_rows_beside_an_infinite_weight(dtype, M, V, D):
    """A token masked by -inf leaves the others' gradients as they are, and padded rows take no part: 0 times
    it is none of theirs."""
    x, w, keep, targets, dloss = masked(M, M, V, D, dtype, torch.arange(V) % 100 == 99, -INF)
    padded = torch.arange(M) % 3 == 1
    targets = torch.where(padded, torch.where(torch.arange(M) % 2 == 1, -1, V), targets)
    x[padded] = float("nan")
    got = run(x, w, targets, dloss, None)
    x[padded] = 0.0
    on = ~padded.cuda()
    assert (got["dx"][~on] == 0).all()
    got["lse"][~on] = 0.0
    where = torch.full((V,), -100)
    where[keep] = torch.arange(len(keep))
    want = ref.head(x[~padded], w[keep], where[targets[~padded]], 1.0, dloss[~padded])
    for k in ("loss", "lse"):
        check(got[k][on], want[k], k)
    check(got["dx"][on][:, 1:], [v[:, 1:] for v in want["dx"]], "dx")
    check(got["dweight"][keep.cuda()], want["dweight"], "dweight")
    hidden = torch.ones(V, dtype=torch.bool, device="cuda")
    hidden[keep] = False
    assert (got["dweight"][hidden] == 0).all()
    # a weight of NaN makes every other row NaN
    w[0] = float("nan")
    got = run(x, w, targets, dloss, None)
    assert (got["dx"][~on] == 0).all() and (got["loss"][~on] == 0).all() and got["dx"][on].isnan().all()
