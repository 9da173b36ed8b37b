"""The gated recurrence and the block norms as they are used: a block's forward
and backward end to end, beside the operators that were there before; two
streams at once, captured and replayed graphs, workspaces of the caller."""
from __future__ import annotations

import numpy as np
import pytest

import block_ref as ref
import mamba_selective_scan_causal_amd as mss
from block_util import back, gated_inputs, put, to_gpu
from gpu_util import announce

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


def block_forward(p, tokens, stream, B, L):
    """x -> norm + projections -> conv1d_silu -> gated_scan with gate -> gated_norm into the
    residual stream, in fp32; returns the new stream and what the backward pass needs."""
    n, s = mss.add_norm(tokens, stream, p["w1"], alpha=0.5)
    proj = n @ p["proj"]                                             # u | r | i | z
    D = proj.shape[1] // 4
    u, r, i, z = proj.split(D, 1)
    c = mss.conv1d_silu(u.contiguous(), p["w_conv"], batch=B, seq_len=L)
    y, ck, hl = mss.gated_scan(c, r, i, p["decay"], z, batch=B, seq_len=L, gate="decay", h_ckpt=True, h_last=True)
    o = y @ p["out"]
    out = mss.gated_norm(o, None, p["w2"], residual=s, scale=p["scale"], alpha=0.5)
    return out, hl, dict(n=n, s=s, u=u.contiguous(), r=r, i=i, z=z, c=c, ck=ck, y=y, o=o)


def block_backward(p, k, dout, B, L):
    g = {}
    after = mss.gated_norm_backward(k["o"], None, p["w2"], None, p["scale"], dout, alpha=0.5)
    g["w2"], g["scale"] = after["dweight"], after["dscale"]
    g["out"] = k["y"].t().contiguous() @ after["dx"]
    dy = after["dx"] @ p["out"].t().contiguous()
    D = dy.shape[1]
    dproj = torch_empty(dy.shape[0], 4 * D)
    _, dr, di, dz = dproj.split(D, 1)
    scan = mss.gated_scan_backward(k["c"], k["r"], k["i"], p["decay"], k["z"], None, k["ck"], dy, batch=B, seq_len=L,
                                   gate="decay", out=dict(dr=dr, di=di, dz=dz))
    g["decay"] = scan["ddecay"]
    du, g["w_conv"], _ = mss.conv1d_silu_backward(k["u"], p["w_conv"], None, scan["dx"], batch=B, seq_len=L)
    dproj[:, :D] = du
    g["proj"] = k["n"].t().contiguous() @ dproj
    dn = dproj @ p["proj"].t().contiguous()
    first = mss.add_norm_backward(k["s"], p["w1"], dn, dout, alpha=0.5)
    g["w1"] = first["dweight"]
    return g, first["dx"], first["dresidual"]


def torch_empty(*shape):
    import torch
    return torch.empty(shape, device="cuda")


def block_exact(p, tokens, stream, B, L):
    """The same block in torch float64, differentiable."""
    import torch
    s = stream + 0.5 * tokens
    norm = lambda v, w: v * (v.pow(2).mean(-1, keepdim=True) + 1e-6).rsqrt() * w
    proj = norm(s, p["w1"]) @ p["proj"]
    D = proj.shape[1] // 4
    u, r, i, z = (t.reshape(B, L, D) for t in proj.split(D, 1))
    K = p["w_conv"].shape[1]
    pad = torch.cat([torch.zeros_like(u[:, :K - 1]), u], 1)
    c = torch.nn.functional.silu(sum(p["w_conv"][:, t] * pad[:, K - 1 - t:K - 1 - t + L] for t in range(K)))
    la = -8.0 * torch.nn.functional.softplus(p["decay"]) * torch.sigmoid(r)
    a, v = la.exp(), (-torch.expm1(2 * la)).sqrt() * torch.sigmoid(i) * c
    h, hs = torch.zeros_like(v[:, 0]), []
    for t in range(L):
        h = a[:, t] * h + v[:, t]
        hs.append(h)
    y = (torch.stack(hs, 1) * torch.nn.functional.silu(z)).reshape(B * L, D)
    return s + 0.5 * p["scale"] * norm(y @ p["out"], p["w2"]), h


@pytest.mark.parametrize("B,L,W,D", [(2, 75, 24, 40), (1, 300, 33, 70)])
def test_a_block_forward_and_backward(B, L, W, D):
    """Against the block in float64 with autograd.  Each value passes about ten operators and three
    matrix products of at most 280 terms, each worth K = 64 half steps of its largest terms: 1e-4 of
    the tensor's rms (12 * 64 * 2^-24 = 4.6e-5, and twice that for the sums over rows)."""
    import torch
    rng = np.random.default_rng(B + L)
    n = lambda *s, sd=1.0, m=0.0: put(rng.normal(m, sd, size=s))
    p = dict(w1=n(W, sd=0.1, m=1), proj=n(W, 4 * D, sd=W ** -0.5), w_conv=n(D, 4, sd=0.5), decay=n(D, m=-3),
             out=n(D, W, sd=D ** -0.5), w2=n(W, sd=0.1, m=1), scale=n(W, sd=0.1, m=1))
    tokens, stream, dout = n(B * L, W), n(B * L, W), n(B * L, W)
    out, hl, kept = block_forward(p, tokens, stream, B, L)
    g, dtokens, dstream = block_backward(p, kept, dout, B, L)
    torch.cuda.synchronize()
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    t64, s64 = tokens.double().requires_grad_(), stream.double().requires_grad_()
    want, h64 = block_exact(q, t64, s64, B, L)
    want.backward(dout.double())
    pairs = dict(out=(out, want), h_last=(hl, h64), dtokens=(dtokens, t64.grad), dstream=(dstream, s64.grad),
                 **{"d" + k: (g[k], q[k].grad) for k in p})
    for k, (got, exact) in pairs.items():
        exact = exact.detach()
        err = ((got.double() - exact).abs().max() / exact.pow(2).mean().sqrt()).item()
        announce(f"{k} {err:.1e}")
        assert err <= 1e-4, (k, err)


def test_after_the_selective_and_ssd_scans():
    """The gated norm behind the scans that were there before: their ungated outputs, normed with
    the gate, equal the same steps in float64 on those outputs."""
    import torch
    rng = np.random.default_rng(2)
    B, L, H, P, N = 1, 96, 4, 16, 16
    n = lambda *s: put(rng.normal(size=s))
    D, M = H * P, B * L
    x, z, w = n(M, D), n(M, D), n(D)
    ssd, _ = mss.ssd_scan(x, n(M, H), n(H), n(M, N), n(M, N), batch=B, seq_len=L, head_dim=P, d_state=N, disc="euler")
    sel, _, _ = mss.selective_scan(x, n(M, D), n(D, N), n(M, N), n(M, N), batch=B, seq_len=L, disc="zoh")
    for y in (ssd, sel):
        got = mss.gated_norm(y, z, w, groups=H)
        torch.cuda.synchronize()
        val, tol = ref.gated_norm(back(y), back(z), back(w), None, None, None, groups=H, order="before", kind="rms",
                                  eps=1e-6, alpha=1.0)
        assert (np.abs(back(got) - val["y"]) <= tol["y"] + ref.U * np.abs(val["y"])).all()


# ---- streams, graphs, workspaces ----------------------------------------------------------

def scan_case(seed, B, L, D, dtype="bf16", gate="decay"):
    rng = np.random.default_rng(seed)
    a = gated_inputs(rng, B, L, D, gate, z=True, h0=True, reset=True)
    a["dout"], a["dh_last"] = rng.normal(size=(B * L, D)), rng.normal(size=(B, D))
    g, _ = to_gpu(a, dtype)
    return g, dict(batch=B, seq_len=L, gate=gate)


def scan_both(g, kw, **more):
    y, ck, hl = mss.gated_scan(g["x"], g["r"], g["i"], g["decay"], g["z"], g["h0"], g["reset"], h_ckpt=True,
                               h_last=True, **kw, **more)
    gr = mss.gated_scan_backward(g["x"], g["r"], g["i"], g["decay"], g["z"], g["reset"], ck, g["dout"],
                                 dh_last=g["dh_last"], need_dh0=True, **kw, **more)
    return [y, ck, hl, *(gr[k] for k in sorted(gr) if gr[k] is not None)]


def norm_case(seed, M, D):
    rng = np.random.default_rng(seed)
    n = lambda *s, t="bf16": put(rng.normal(size=s), t)
    return dict(x=n(M, D), z=n(M, D), res=n(M, D, t="f32"), d=n(M, D), w=n(D, t="f32"), s=n(D, t="f32"))


def norm_both(c, **more):
    y, s = mss.add_norm(c["x"], c["res"], c["w"], scale=c["s"], **more)
    a = mss.add_norm_backward(s, c["w"], c["d"], c["res"], c["x"], c["s"], bias=True, **more)
    o = mss.gated_norm(c["x"], c["z"], c["w"], groups=2, **more)
    b = mss.gated_norm_backward(c["x"], c["z"], c["w"], None, c["s"], c["d"], groups=2, **more)
    return [y, s, o, *(a[k] for k in sorted(a) if a[k] is not None), *(b[k] for k in sorted(b) if b[k] is not None)]


def test_two_streams_at_once():
    import torch
    ga, ka = scan_case(1, 2, 3000, 300)
    gb, kb = scan_case(2, 3, 1700, 192, "f32", "decay")
    na, nb = norm_case(3, 900, 1536), norm_case(4, 700, 520)
    want = [scan_both(ga, ka), scan_both(gb, kb), norm_both(na), norm_both(nb)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(3):
        for s, (g, k, n) in ((s1, (ga, ka, na)), (s2, (gb, kb, nb))):
            with torch.cuda.stream(s):
                got.append((scan_both(g, k), norm_both(n)))
    torch.cuda.synchronize()
    for j, (scan, norm) in enumerate(got):
        assert all(torch.equal(p, q) for p, q in zip(scan, want[j % 2]))
        assert all(torch.equal(p, q) for p, q in zip(norm, want[2 + j % 2]))


def test_stream_argument():
    """Work on a stream that is not the current one, workspaces allocated by the call."""
    import torch
    g, k = scan_case(5, 1, 2000, 130)
    n = norm_case(6, 300, 640)
    want = scan_both(g, k), norm_both(n)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = scan_both(g, k, stream=s), norm_both(n, stream=s)
    junk = [torch.full((1 << 18,), 7.0, device="cuda") for _ in range(8)]     # what reuse would hit
    torch.cuda.synchronize()
    for p, q in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(p, q))
    assert all((j == 7).all() for j in junk)


def test_graph_replay():
    """A captured forward and backward replays to the eager bits, again after the inputs changed,
    with eager calls on the same inputs between the replays."""
    import torch
    g, k = scan_case(7, 2, 1500, 200)
    n = norm_case(8, 333, 768)
    want = scan_both(g, k) + norm_both(n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = scan_both(g, k) + norm_both(n)
    for _ in range(3):
        for t in got:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        scan_both(g, k)
    g["x"].mul_(-0.5)
    n["x"].mul_(2)
    want = scan_both(g, k) + norm_both(n)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_graph_of_decoding_steps():
    """64 single-token steps with the state carried inside the graph."""
    import torch
    g, _ = scan_case(9, 4, 64, 256)
    rows = [torch.arange(4, device="cuda") * 64 + t for t in range(64)]
    tok = [{k: g[k][r].contiguous() for k in ("x", "r", "i", "z")} for r in rows]

    def steps(h):
        return [mss.gated_step(t["x"], t["r"], t["i"], g["decay"], t["z"], h, gate="decay") for t in tok]

    h = g["h0"].clone()
    want = steps(h)
    torch.cuda.synchronize()
    final = h.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = steps(h)
    for _ in range(3):
        h.copy_(g["h0"])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, final) and all(torch.equal(p, q) for p, q in zip(got, want))


def test_callers_workspace_with_anything_in_it():
    """One workspace for calls in a row, larger than needed, misaligned by a byte, and full of what
    the last call (or nobody) left there: the same bits; the bytes behind the reported size stay."""
    import torch
    g, k = scan_case(10, 2, 1400, 130)
    D = 130
    want = scan_both(g, k)
    torch.cuda.synchronize()
    need = max(mss.gated_workspace_bytes(op, batch=2, seq_len=1400, d_inner=D, gate="decay")
               for op in (mss.OP_GATED_SCAN, mss.OP_GATED_SCAN_BACKWARD))
    for fill in (0, 255, 127):
        ws = torch.full((need + 1024 + 1,), fill, dtype=torch.uint8, device="cuda")[1:]
        for _ in range(2):
            got = scan_both(g, k, workspace=ws)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert (ws[need + 512:] == fill).all()
    c = norm_case(11, 200, 520)
    want = mss.gated_norm_backward(c["x"], c["z"], c["w"], None, c["s"], c["d"])
    need = mss.norm_workspace_bytes(mss.OP_GATED_NORM_BACKWARD, rows=200, width=520)
    ws = torch.full((need + 1024,), 255, dtype=torch.uint8, device="cuda")
    got = mss.gated_norm_backward(c["x"], c["z"], c["w"], None, c["s"], c["d"], workspace=ws)
    torch.cuda.synchronize()
    assert all(got[k] is None or torch.equal(got[k], want[k]) for k in want)
    assert (ws[need + 512:] == 255).all()
    with pytest.raises(mss.MssError) as err:
        mss.gated_norm_backward(c["x"], c["z"], c["w"], None, c["s"], c["d"], workspace=ws[:need // 2])
    assert err.value.status == -4
