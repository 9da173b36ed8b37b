"""The embedding, the head's loss and clipping as they are used: a model's training step with a tied
table around a block of the library, two streams at once, captured and replayed graphs, workspaces
of the caller, scoring in pieces."""
from __future__ import annotations

import pytest
import torch

import mamba_selective_scan_causal_amd as mss
from ends_util import TYPES, generator, normal, some_ids
from gpu_util import announce

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


# ---- a training step --------------------------------------------------------------------------

def step(p, ids, targets, B, L, max_norm):
    """tokens -> norm -> gated scan -> norm -> head, tied to the table; the loss and the clipped gradients."""
    x = mss.embedding(ids, p["table"], scale=2.0)
    n1, s1 = mss.add_norm(x, None, p["w1"])
    r, z = (n1 @ p["proj"]).split(n1.shape[1], 1)
    y, ck, _ = mss.gated_scan(n1, r, None, None, z, batch=B, seq_len=L, gate="sigmoid", h_ckpt=True)
    n2, s2 = mss.add_norm(y, s1, p["w2"])
    loss, lse = mss.head_loss(n2, p["table"], targets, logit_scale=0.5)
    V = p["table"].shape[0]
    valid = ((targets >= 0) & (targets < V)).float()
    dloss = valid / valid.sum()
    g = {}
    head = mss.head_loss_backward(n2, p["table"], targets, lse, dloss, logit_scale=0.5)
    b2 = mss.add_norm_backward(s2, p["w2"], head["dx"])
    g["w2"] = b2["dweight"]
    scan = mss.gated_scan_backward(n1, r, None, None, z, None, ck, b2["dx"], batch=B, seq_len=L, gate="sigmoid")
    dproj = torch.cat([scan["dr"], scan["dz"]], 1)
    g["proj"] = n1.t().contiguous() @ dproj
    dn1 = scan["dx"] + dproj @ p["proj"].t().contiguous()
    b1 = mss.add_norm_backward(s1, p["w1"], dn1, b2["dresidual"])
    g["w1"] = b1["dweight"]
    g["table"] = mss.embedding_backward(ids, b1["dx"], vocab=V, scale=2.0, accumulate=True, out=head["dweight"])
    names = sorted(g)
    _, norm = mss.clip_grads([g[k] for k in names], max_norm)
    return (loss * dloss).sum(), norm, g


def step_exact(p, ids, targets, B, L):
    V = p["table"].shape[0]
    inside = (ids >= 0) & (ids < V)
    x = torch.where(inside[:, None], 2.0 * p["table"][ids.clamp(0, V - 1)], 0.0)
    norm = lambda v, w: v * (v.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt() * w
    n1, s1 = norm(x, p["w1"]), x
    r, z = (n1 @ p["proj"]).split(n1.shape[1], 1)
    a = torch.sigmoid(r).reshape(B, L, -1)
    v = (1 - a) * n1.reshape(B, L, -1)
    h, hs = torch.zeros_like(v[:, 0]), []
    for t in range(L):
        h = a[:, t] * h + v[:, t]
        hs.append(h)
    y = torch.stack(hs, 1).reshape(B * L, -1) * torch.nn.functional.silu(z)
    n2 = norm(s1 + y, p["w2"])
    logits = 0.5 * (n2 @ p["table"].t())
    return torch.nn.functional.cross_entropy(logits, torch.where((targets >= 0) & (targets < V), targets, -100))


@pytest.mark.parametrize("max_norm", [1e9, 1e-3])
def test_a_training_step_with_a_tied_table(max_norm):
    """Against the step in float64 with autograd.  About ten operators and four products of at most
    140 terms (37 for the head's D), each worth K = 64 half steps of its largest terms, as for a block:
    14 * 64 * 2^-24 = 5.3e-5, and twice that for the sums over rows and tokens: 1e-4 of a tensor's rms."""
    B, L, D, V = 2, 70, 36, 150
    g = generator(1)
    p = dict(table=normal(g, V, D, std=0.5), w1=normal(g, D, std=0.1) + 1, w2=normal(g, D, std=0.1) + 1,
             proj=normal(g, D, 2 * D, std=D ** -0.5))
    ids, targets = some_ids(g, B * L, V), some_ids(g, B * L, V)
    loss, norm, grads = step({k: v.cuda() for k, v in p.items()}, ids.cuda(), targets.cuda(), B, L, max_norm)
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    want = step_exact(q, ids, targets, B, L)
    want.backward()
    total = sum(v.grad.pow(2).sum() for v in q.values()).sqrt()
    factor = min(1.0, max_norm / total.item())
    assert abs(loss.item() - want.item()) <= 1e-4 * want.item()
    assert abs(norm.item() - total.item()) <= 1e-4 * total.item()
    for k, v in q.items():
        e = v.grad * factor
        err = ((grads[k].double().cpu() - e).abs().max() / e.pow(2).mean().sqrt()).item()
        announce(f"{k} {err:.1e}")
        assert err <= 1e-4, (k, err)


def test_scoring_in_pieces_of_a_prompt():
    """Rows scored a few at a time have the scores they have together, to the products' order."""
    g = generator(2)
    M, V, D = 300, 1000, 128
    x, w, t = normal(g, M, D, dtype=torch.bfloat16).cuda(), normal(g, V, D, std=0.1, dtype=torch.bfloat16).cuda(), \
        some_ids(g, M, V).cuda()
    loss, lse = mss.head_loss(x, w, t)
    for size in (1, 7, 64, 129):
        parts = [mss.head_loss(x[i:i + size], w, t[i:i + size]) for i in range(0, M, size)]
        for whole, k in ((loss, 0), (lse, 1)):
            got = torch.cat([q[k] for q in parts])
            # logits of order 1, log sums of order 10: sums of 128 products and of 1000 exponentials
            assert (got - whole).abs().max() <= 2e-5


def test_a_shard_of_the_vocabulary():
    """Two halves of the table: the lookups add up to the whole's, the gradients are the whole's rows,
    and the loss follows from the halves' log sums and target logits."""
    g = generator(3)
    M, V, D = 200, 500, 64
    x, w, t = normal(g, M, D).cuda(), normal(g, V, D, std=0.2).cuda(), torch.randint(0, V, (M,), generator=g).cuda()
    h = V // 2
    assert torch.equal(mss.embedding(t, w), mss.embedding(t, w[:h]) + mss.embedding(t - h, w[h:]))
    dw = mss.embedding_backward(t, x, vocab=V)
    assert torch.equal(dw[:h], mss.embedding_backward(t, x, vocab=h))
    assert torch.equal(dw[h:], mss.embedding_backward(t - h, x, vocab=V - h))
    loss, lse = mss.head_loss(x, w, t)
    (la, sa), (lb, sb) = mss.head_loss(x, w[:h], t), mss.head_loss(x, w[h:], t - h)
    both = torch.logaddexp(sa, sb)
    own = torch.where(t < h, sa - la, sb - lb)
    assert (both - lse).abs().max() <= 1e-5 and (both - own - loss).abs().max() <= 1e-5


# ---- streams, graphs, workspaces ----------------------------------------------------------------

def make(seed, M=700, V=900, D=96, dtype="bf16"):
    g = generator(seed)
    t = TYPES[dtype]
    c = dict(ids=some_ids(g, M, V), w=normal(g, V, D, std=0.2, dtype=t), dy=normal(g, M, D, dtype=t),
             x=normal(g, M, D, dtype=t), targets=some_ids(g, M, V), dloss=normal(g, M, std=1 / M),
             g1=normal(g, 40001, dtype=t), g2=normal(g, 33, 70))
    return {k: v.cuda() for k, v in c.items()}


def everything(c, **more):
    V = c["w"].shape[0]
    y = mss.embedding(c["ids"], c["w"], **more)
    dw = mss.embedding_backward(c["ids"], c["dy"], vocab=V, **({k: v for k, v in more.items()}))
    loss, lse = mss.head_loss(c["x"], c["w"], c["targets"], **more)
    g = mss.head_loss_backward(c["x"], c["w"], c["targets"], lse, c["dloss"], **more)
    out = [torch.empty_like(c["g1"]), torch.empty_like(c["g2"])]
    out, norm = mss.clip_grads([c["g1"], c["g2"]], 1.0, out=out, **more)
    return [y, dw, loss, lse, g["dx"], g["dweight"], *out, norm]


def test_two_streams_at_once():
    a, b = make(4), make(5, 1100, 400, 71, "f32")
    want = [everything(a), everything(b)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(3):
        for s, c in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append(everything(c))
    torch.cuda.synchronize()
    for j, r in enumerate(got):
        assert all(torch.equal(p, q) for p, q in zip(r, want[j % 2]))


@pytest.mark.parametrize("call", ["embedding", "embedding_backward", "head_loss", "head_loss_backward", "clip_grads"])
def test_stream_argument(call):
    """A call on a stream that is not the current one, its memory its own: junk allocated on the
    current stream right after stays as it is, and so does what the call returns."""
    c = make(6)
    V = c["w"].shape[0]
    _, lse = mss.head_loss(c["x"], c["w"], c["targets"])
    calls = {
        "embedding": lambda **k: [mss.embedding(c["ids"], c["w"], **k)],
        "embedding_backward": lambda **k: [mss.embedding_backward(c["ids"], c["dy"], vocab=V, **k)],
        "head_loss": lambda **k: list(mss.head_loss(c["x"], c["w"], c["targets"], **k)),
        "head_loss_backward": lambda **k: list(mss.head_loss_backward(c["x"], c["w"], c["targets"], lse, c["dloss"],
                                                                      **k).values()),
        "clip_grads": lambda **k: [mss.clip_grads([c["g1"].clone(), c["g2"].clone()], 1.0)[1], mss.grad_norm(
            [c["g1"], c["g2"]], **k)],
    }
    want = calls[call]()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = calls[call](stream=s)
    junk = [torch.full((1 << 18,), 7.0, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert all((j == 7).all() for j in junk)


def test_graph_replay():
    """Captured once, replayed with eager calls and other values between, each time the eager bits."""
    a = make(7)
    want = everything(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything(a)
    for _ in range(3):
        for t in got:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        everything(a)
    a["x"].mul_(-0.5)
    a["ids"].copy_(a["ids"].flip(0))
    a["targets"].copy_(a["targets"].roll(5))
    a["g1"].mul_(3)
    want = everything(a)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_two_graphs_with_a_workspace_each():
    """Two captured backward passes on two streams at once, each with a workspace of its own."""
    cases, graphs, got, want = [make(8), make(9, 900, 1200, 64)], [], [], []
    kept = []                     # what the graphs read and write has to live as long as they do
    for c in cases:
        _, lse = mss.head_loss(c["x"], c["w"], c["targets"])
        M, (V, D) = c["x"].shape[0], c["w"].shape
        need = max(mss.head_workspace_bytes(mss.OP_HEAD_LOSS_BACKWARD, rows=M, vocab=V, width=D, dtype=torch.bfloat16),
                   mss.embed_workspace_bytes(rows=M, vocab=V, width=D))
        ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")

        def both(c=c, lse=lse, ws=ws, V=V):
            g = mss.head_loss_backward(c["x"], c["w"], c["targets"], lse, c["dloss"], workspace=ws)
            return [g["dx"], mss.embedding_backward(c["ids"], c["dy"], vocab=V, accumulate=True, out=g["dweight"],
                                                    workspace=ws)]
        kept.append((lse, ws, both))
        want.append(both())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got.append(both())
        graphs.append(graph)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(g, w))


def test_callers_workspace_with_anything_in_it():
    """One workspace for all calls in a row, off by a byte and full of anything: the same bits, and the
    bytes behind the reported size stay."""
    c = make(10, dtype="f16")
    M, (V, D) = c["x"].shape[0], c["w"].shape
    want = everything(c)
    needs = [mss.embed_workspace_bytes(rows=M, vocab=V, width=D), mss.clip_workspace_bytes(2)] + [
        mss.head_workspace_bytes(op, rows=M, vocab=V, width=D, dtype=torch.float16)
        for op in (mss.OP_HEAD_LOSS, mss.OP_HEAD_LOSS_BACKWARD)]
    for fill in (0, 255, 127):
        ws = torch.full((max(needs) + 1024 + 1,), fill, dtype=torch.uint8, device="cuda")[1:]
        dw = mss.embedding_backward(c["ids"], c["dy"], vocab=V, workspace=ws)
        loss, lse = mss.head_loss(c["x"], c["w"], c["targets"], workspace=ws)
        g = mss.head_loss_backward(c["x"], c["w"], c["targets"], lse, c["dloss"], workspace=ws)
        out, norm = mss.clip_grads([c["g1"].clone(), c["g2"].clone()], 1.0, workspace=ws)
        got = [want[0], dw, loss, lse, g["dx"], g["dweight"], *out, norm]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert (ws[max(needs) + 512:] == fill).all()
    small = torch.empty(max(needs), dtype=torch.uint8, device="cuda")
    for need, call in ((needs[0], lambda w: mss.embedding_backward(c["ids"], c["dy"], vocab=V, workspace=w)),
                       (needs[1], lambda w: mss.grad_norm([c["g1"], c["g2"]], workspace=w)),
                       (needs[2], lambda w: mss.head_loss(c["x"], c["w"], c["targets"], workspace=w))):
        with pytest.raises(mss.MssError) as err:
            call(small[:need // 2])
        assert err.value.status == -4


def test_refusals():
    c = make(11)
    V = c["w"].shape[0]
    bad = [
        (TypeError, lambda: mss.embedding(c["ids"].float(), c["w"])),
        (TypeError, lambda: mss.embedding(c["ids"], c["w"], out_dtype=torch.float16)),
        (ValueError, lambda: mss.embedding(c["ids"].reshape(2, -1), c["w"])),
        (ValueError, lambda: mss.embedding(c["ids"].cpu(), c["w"])),
        (ValueError, lambda: mss.embedding(c["ids"][::2], c["w"])),
        (ValueError, lambda: mss.embedding(c["ids"], c["w"], out=torch.empty(3, 96, device="cuda", dtype=torch.bfloat16))),
        (ValueError, lambda: mss.embedding(c["ids"], c["w"].t())),
        (ValueError, lambda: mss.embedding_backward(c["ids"], c["dy"], vocab=V, accumulate=True)),
        (ValueError, lambda: mss.embedding_backward(c["ids"], c["dy"], vocab=-1)),
        (ValueError, lambda: mss.embedding_backward(c["ids"], c["dy"][1:], vocab=V)),
        (TypeError, lambda: mss.embedding_backward(c["ids"], c["dy"], vocab=V, dtype=torch.float16)),
        (TypeError, lambda: mss.head_loss(c["x"].float(), c["w"], c["targets"])),
        (ValueError, lambda: mss.head_loss(c["x"][:, 1:], c["w"], c["targets"])),
        (ValueError, lambda: mss.head_loss(c["x"], c["w"], c["targets"][1:])),
        (TypeError, lambda: mss.head_loss(c["x"], c["w"], c["targets"].short())),
        (TypeError, lambda: mss.head_loss_backward(c["x"], c["w"], c["targets"], c["dloss"], c["dloss"].double())),
        (ValueError, lambda: mss.head_loss_backward(c["x"], c["w"], c["targets"], c["dloss"], None)),
        (ValueError, lambda: mss.head_loss_backward(c["x"], c["w"], c["targets"], c["dloss"], c["dloss"], out=dict(dy=1))),
        (mss.MssError, lambda: mss.embedding(c["ids"], c["w"], scale=float("nan"))),
        (mss.MssError, lambda: mss.embedding(c["ids"], c["w"], out=c["w"][:700])),
        (mss.MssError, lambda: mss.head_loss(c["x"], c["w"], c["targets"], logit_scale=float("inf"))),
        (mss.MssError, lambda: mss.head_loss(c["x"], c["w"][:0], c["targets"])),
        (mss.MssError, lambda: mss.head_loss_backward(c["x"], c["w"], c["targets"], c["dloss"], c["dloss"],
                                                      out=dict(dx=c["x"]))),
    ]
    for k, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            raise AssertionError(f"case {k} was taken")
