"""The two ends of a model around its blocks, and the step before the update: cases, plain forms, exact values.

Embedding (``embedding``, ``embedding_backward``), for rows m of tokens and a table W (V, D)
    y_m  = scale W[id_m]                          (zeros where id_m is not in 0 .. V-1)
    dW_v = scale sum_{m: id_m = v} dy_m           (written, or added to what is there)

Head and loss (``head_loss``, ``head_loss_backward``), for rows x_m and a head W (V, D)
    l_mv   = s x_m . W_v,   lse_m = log sum_v exp(l_mv)
    loss_m = lse_m - l_{m,t_m}                    (0 where t_m is not in 0 .. V-1: an ignored row)
    dl_mv  = (dloss_m + dlse_m) exp(l_mv - lse_m) - dloss_m [v = t_m]      (0 in ignored rows)
    dx     = s dl W,   dW = s dl^T x

Clipping (``grad_norm``, ``clip_grads``), over a list of tensors g
    norm = scale sqrt(sum g^2),   out = g scale min(1, max_norm / norm)    (out = g where norm is not finite)
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
Z_LOSS = 1e-4
MAX_NORM = 1.0
EMBED_SCALE = 0.75
HEAD_SCALE = 0.5
MOST = 16384 * 65536 * 2560      # rows * vocabulary * width of the largest head


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # decoding for a few users: the rows of their last tokens
        dict(name="embed_tokens", op="embed", dtype="bf16", out="f32", rows=4, d=1536, vocab=32768),
        # a few prompts of odd length and width, some of them padded
        dict(name="embed_prompts", op="embed", dtype="f16", out="f16", rows=1551, d=1001, vocab=10007),
        # a training step: the lookup into a 32-bit residual stream, and the table's gradient
        dict(name="embed_train", op="embed_train", dtype="bf16", out="f32", rows=32768, d=2560, vocab=65536),
        # a table tied to the head: the tokens' gradient is added to the head's
        dict(name="embed_tied", op="embed_tied", dtype="bf16", out="bf16", rows=16384, d=1536, vocab=32768),
        # scores of a few drafted tokens
        dict(name="head_tokens", op="head", dtype="bf16", rows=8, d=2560, vocab=65536),
        # scores of a prompt, odd sizes
        dict(name="head_prompt", op="head", dtype="bf16", rows=517, d=1536, vocab=50021),
        # a training step's loss and all its gradients
        dict(name="head_train", op="head_train", dtype="bf16", rows=8192, d=1536, vocab=32768, z_loss=False),
        # the same at the large width and vocabulary, with a penalty on the log of the sum
        dict(name="head_train_large", op="head_train", dtype="bf16", rows=16384, d=2560, vocab=65536, z_loss=True),
        # ragged sizes of everything
        dict(name="head_train_odd", op="head_train", dtype="f16", rows=1551, d=1001, vocab=10007, z_loss=False),
        # in 32 bits
        dict(name="head_train_f32", op="head_train", dtype="f32", rows=2048, d=768, vocab=32768, z_loss=False),
        # one block's gradients, summed over two micro-batches, clipped in place
        dict(name="clip_block", op="clip", dtype="f32", width=768, layers=1, vocab=0, scale=0.5, inplace=True),
        # the gradients of a table and several wide blocks in 16 bits, clipped into the buffers of the update
        dict(name="clip_model", op="clip", dtype="bf16", width=2560, layers=6, vocab=65536, scale=1.0,
             inplace=False),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(max(low, high))))))


def draw(rng):
    op = rng.choice(["embed", "embed_train", "embed_tied", "head", "head", "head_train", "head_train", "clip"])
    dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
    if op == "clip":
        inplace = rng.random() < 0.5
        return dict(op=op, dtype=dtype, width=_log_int(rng, 64, 2560), layers=_log_int(rng, 1, 6),
                    vocab=rng.choice([0, _log_int(rng, 1000, 65536)]), scale=0.5 if inplace else rng.choice([1.0, 0.125]),
                    inplace=inplace)
    d = _log_int(rng, 32, 2560)
    if rng.random() < 0.6:
        d = max(8, d // 8 * 8)
    vocab = _log_int(rng, 500, 65536)
    if op.startswith("embed"):
        return dict(op=op, dtype=dtype, out=dtype if op == "embed_tied" else rng.choice([dtype, "f32"]),
                    rows=_log_int(rng, 1, 32768), d=d, vocab=vocab)
    # 32-bit products run at a tenth of the rate
    most = MOST // (16 if dtype == "f32" else 2)
    rows = _log_int(rng, 1, min(16384, most // (vocab * d)))
    return dict(op=op, dtype=dtype, rows=rows, d=d, vocab=vocab, **(
        dict(z_loss=rng.random() < 0.3) if op == "head_train" else {}))


# ----------------------------------------------------------------- the inputs

def _token_weights(vocab):
    """How often tokens occur, by rank: the usual falling law of text."""
    w = 1.0 / (np.arange(vocab) + 2.7)
    return w / w.sum()


def _clip_shapes(width, layers, vocab):
    """Parameters of a block: projections, convolution, state matrix, skip, norms; and the table."""
    inner, rank, state = 2 * width, -(-width // 16), 16
    block = [(2 * inner, width), (inner, 4), (inner,), (rank + 2 * state, inner), (inner, rank), (inner,),
             (inner, state), (inner,), (width, inner), (width,)]
    return block * layers + [(width,)] + ([(vocab, width)] if vocab else [])


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 29)
    t = DTYPES[case["dtype"]]
    s = dict(case=dict(case))

    def normal(*shape, std=1.0, dtype=t):
        return torch.empty(shape, dtype=torch.float32, device="cuda").normal_(0, std, generator=g).to(dtype)

    def uniform(n):
        return torch.empty(n, dtype=torch.float64, device="cuda").uniform_(0, 1, generator=g)

    if case["op"] == "clip":
        # sizes that differ from tensor to tensor; vectors held in 32 bits
        s["grads"] = [normal(*shape, std=10.0 ** (-3 - k % 3), dtype=t if len(shape) == 2 else torch.float32)
                      for k, shape in enumerate(_clip_shapes(case["width"], case["layers"], case["vocab"]))]
        s["out"] = s["grads"] if case["inplace"] else [torch.empty_like(v) for v in s["grads"]]
        return s
    rows, d, vocab = case["rows"], case["d"], case["vocab"]

    def tokens(away):
        share = torch.from_numpy(np.cumsum(_token_weights(vocab))).cuda()
        rank = torch.searchsorted(share, uniform(rows)).clamp_(max=vocab - 1)
        ids = torch.randperm(vocab, generator=g, device="cuda")[rank]
        return torch.where(uniform(rows) < away, -100, ids)          # padding

    if case["op"].startswith("embed"):
        s["ids"] = tokens(0.05)
        s["weight"] = normal(vocab, d, std=0.02)
        if case["op"] != "embed":
            s["dy"] = normal(rows, d, std=1e-2, dtype=DTYPES[case["out"]])
        if case["op"] == "embed_tied":
            s["dweight"] = normal(vocab, d, std=1e-2)
        return s
    s["weight"] = normal(vocab, d, std=2.0 * d ** -0.5)
    s["targets"] = tokens(0.1)
    # normed rows that lean to their target by any amount, as a half-trained model's do
    lean = (uniform(rows) * 6.0).float()[:, None]
    s["x"] = (normal(rows, d, dtype=torch.float32) + lean * s["weight"][s["targets"].clamp(min=0)].float()).to(t)
    if case["op"] == "head_train":
        valid = (s["targets"] >= 0).float()
        s["dloss"] = valid / valid.sum().clamp(min=1.0)
    return s


# --------------------------------------------------------------- the one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import mamba_selective_scan_causal_amd as mss
    c = s["case"]
    op = c["op"]
    if op == "clip":
        out, norm = mss.clip_grads(s["grads"], MAX_NORM, scale=c["scale"], out=s["out"])
        return dict(out=out, norm=norm)
    if op == "embed_tied":
        return dict(dweight=mss.embedding_backward(s["ids"], s["dy"], vocab=c["vocab"], scale=EMBED_SCALE,
                                                   accumulate=True, out=s["dweight"]))
    if op.startswith("embed"):
        y = mss.embedding(s["ids"], s["weight"], scale=EMBED_SCALE, out_dtype=DTYPES[c["out"]])
        if op == "embed":
            return dict(y=y)
        return dict(y=y, dweight=mss.embedding_backward(s["ids"], s["dy"], vocab=c["vocab"], scale=EMBED_SCALE,
                                                        dtype=s["weight"].dtype))
    loss, lse = mss.head_loss(s["x"], s["weight"], s["targets"], logit_scale=HEAD_SCALE)
    if op == "head":
        return dict(loss=loss, lse=lse)
    grads = mss.head_loss_backward(s["x"], s["weight"], s["targets"], lse, s["dloss"], _dlse(s, c, lse),
                                   logit_scale=HEAD_SCALE)
    return dict(grads, loss=loss, lse=lse)


def _dlse(s, c, lse):
    """The gradient that a penalty Z_LOSS lse^2 on each valid row sends to lse."""
    return s["dloss"] * (2.0 * Z_LOSS) * lse if c["z_loss"] else None


# ------------------------------------------------------------ the plain forms

def _plain(s):
    c = s["case"]
    return (_plain_clip if c["op"] == "clip" else _plain_embed if c["op"].startswith("embed") else _plain_head)(s, c)


def _plain_embed(s, c):
    ids, vocab = s["ids"], c["vocab"]
    valid = ((ids >= 0) & (ids < vocab))[:, None]
    at = ids.clamp(0, vocab - 1)
    out = {}
    if c["op"] != "embed_tied":
        y = EMBED_SCALE * s["weight"][at].float()
        out["y"] = torch.where(valid, y, torch.zeros_like(y)).to(DTYPES[c["out"]])
    if c["op"] == "embed":
        return out
    dy = torch.where(valid, s["dy"].double(), 0.0)
    dw = EMBED_SCALE * torch.zeros(vocab, c["d"], dtype=torch.float64, device=ids.device).index_add_(0, at, dy)
    if c["op"] == "embed_tied":
        return dict(dweight=s["dweight"].copy_(dw + s["dweight"]))
    return dict(out, dweight=dw.to(s["weight"].dtype))


def _plain_head(s, c):
    t, w, x = s["targets"], s["weight"].float(), s["x"].float()
    valid = (t >= 0) & (t < c["vocab"])
    at = t.clamp(0, c["vocab"] - 1)[:, None]
    logits = HEAD_SCALE * (x @ w.t())
    top = logits.max(1, keepdim=True).values
    lse = top + torch.log(torch.exp(logits - top).sum(1, keepdim=True))
    loss = torch.where(valid, (lse - logits.gather(1, at))[:, 0], 0.0)
    if c["op"] == "head":
        return dict(loss=loss, lse=lse[:, 0])
    dlse = _dlse(s, c, lse[:, 0])
    dloss = torch.where(valid, s["dloss"], 0.0)[:, None]
    both = dloss if dlse is None else dloss + torch.where(valid, dlse, 0.0)[:, None]
    dl = torch.exp(logits - lse) * both
    dl = dl.scatter_add(1, at, -dloss)
    x = torch.where(valid[:, None], x, 0.0)
    return dict(loss=loss, lse=lse[:, 0], dx=(HEAD_SCALE * (dl @ w)).to(s["x"].dtype),
                dweight=(HEAD_SCALE * (dl.t() @ x)).to(s["weight"].dtype))


def _plain_clip(s, c):
    square = torch.stack([g.double().square().sum() for g in s["grads"]]).sum()
    norm = c["scale"] * torch.sqrt(square)
    factor = torch.where(torch.isfinite(norm), c["scale"] * torch.clamp(MAX_NORM / norm, max=1.0), 1.0).float()
    return dict(out=[o.copy_(g.float() * factor) for g, o in zip(s["grads"], s["out"])], norm=norm.float())


# --------------------------------------------------- what a pass cannot do without

def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "clip":
        shapes = _clip_shapes(case["width"], case["layers"], case["vocab"])
        size = sum(math.prod(v) * (e if len(v) == 2 else 4) for v in shapes)
        return {"bytes": 2 * size, "flops": 3 * sum(math.prod(v) for v in shapes)}
    m, d, v = case["rows"], case["d"], case["vocab"]
    if case["op"].startswith("embed"):
        eo = SIZE[case["out"]]
        # different tokens among the rows that are not padding
        seen = float((1.0 - (1.0 - _token_weights(v)) ** (0.95 * m)).sum())
        ids, lookup = 8 * m, m * d * eo + seen * d * e
        if case["op"] == "embed":
            return {"bytes": ids + lookup, "flops": m * d}
        if case["op"] == "embed_tied":
            return {"bytes": ids + 0.95 * m * d * eo + 2 * seen * d * e, "flops": m * d}
        return {"bytes": 2 * ids + lookup + 0.95 * m * d * eo + v * d * e, "flops": 2 * m * d}
    ins = (m + v) * d * e + m * 8
    if case["op"] == "head":
        return {"bytes": ins + 8 * m, "flops": 2 * m * v * d}
    # a step's loss lies between the two directions, so both read their inputs; the logits once, not again
    return {"bytes": 2 * ins + 16 * m + (m + v) * d * e, "flops": 6 * m * v * d}


# ------------------------------------------------------------ the exact values

def exact(case, seed):
    """The definition in 64 bits: token by token sums through a sorted order (embedding), the logits of a few
    rows at a time (head), the sum of squares (clipping)."""
    s = prepare(case, seed)
    return (_exact_clip if case["op"] == "clip" else _exact_embed if case["op"].startswith("embed") else
            _exact_head)(s, case)


def _exact_embed(s, c):
    inside = (s["ids"] >= 0) & (s["ids"] < c["vocab"])
    out = {}
    if c["op"] != "embed_tied":
        y = torch.zeros(c["rows"], c["d"], dtype=torch.float64, device="cuda")
        y[inside] = EMBED_SCALE * s["weight"][s["ids"][inside]].double()
        out["y"] = y
    if c["op"] == "embed":
        return out
    ids, order = torch.sort(s["ids"][inside], stable=True)
    dy = s["dy"][inside][order].double()
    which, count = torch.unique_consecutive(ids, return_counts=True)
    start = torch.cumsum(count, 0) - count
    dw = torch.zeros(c["vocab"], c["d"], dtype=torch.float64, device="cuda")
    if c["op"] == "embed_tied":
        dw += s["dweight"].double()
    # the k-th occurrence of every token that has so many; then one sum for each token that has more
    few = 64
    for k in range(min(few, int(count.max()) if len(count) else 0)):
        has = count > k
        dw[which[has]] += EMBED_SCALE * dy[start[has] + k]
    for v, a, n in zip(*(w[count > few].tolist() for w in (which, start, count))):
        dw[v] += EMBED_SCALE * dy[a + few:a + n].sum(0)
    return dict(out, dweight=dw)


def _exact_head(s, c):
    train, rows, vocab = c["op"] == "head_train", c["rows"], c["vocab"]
    w, got = s["weight"].double(), []
    dw = torch.zeros_like(w) if train else None
    for r0 in range(0, rows, 1024):
        cut = slice(r0, min(rows, r0 + 1024))
        x, t = s["x"][cut].double(), s["targets"][cut]
        logits = HEAD_SCALE * torch.mm(x, w.t().contiguous())
        lse = torch.logsumexp(logits, 1)
        inside = torch.nonzero((t >= 0) & (t < vocab))[:, 0]
        loss = torch.zeros_like(lse)
        loss[inside] = lse[inside] - logits[inside, t[inside]]
        part = dict(loss=loss, lse=lse)
        if train:
            up, x, t = s["dloss"][cut][inside].double(), x[inside], t[inside]
            dl = torch.softmax(logits[inside], 1)
            both = up * (1.0 + 2.0 * Z_LOSS * lse[inside]) if c["z_loss"] else up
            dl = dl * both[:, None]
            dl[torch.arange(len(t), device=dl.device), t] -= up
            dx = torch.zeros(lse.shape[0], c["d"], dtype=torch.float64, device=dl.device)
            dx[inside] = HEAD_SCALE * torch.mm(dl, w)
            dw += HEAD_SCALE * torch.mm(dl.t().contiguous(), x)
            part["dx"] = dx
        got.append(part)
    out = {k: torch.cat([p[k] for p in got]) for k in got[0]}
    return dict(out, dweight=dw) if train else out


def _exact_clip(s, c):
    norm = c["scale"] * math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in s["grads"]))
    factor = c["scale"] * (MAX_NORM / norm if norm > MAX_NORM else 1.0) if math.isfinite(norm) else 1.0
    return dict(out=[g.double() * factor for g in s["grads"]], norm=torch.tensor(norm, dtype=torch.float64))
