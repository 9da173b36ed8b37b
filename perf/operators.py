"""The gated linear recurrence and the block norms: cases, plain forms and exact values.

Two families around the core of a recurrent block.

Recurrence (``gated_scan``, ``gated_scan_backward``, ``gated_step``), per channel
    h_t = v_t + a_t h_{t-1}   (the carried part dropped where reset_t is set)
    y_t = h_t SiLU(z_t)       (or h_t)
  with a, v from the token's own gates:
    sigmoid   a = sigma(r)                                 v = (1 - a) x
    decay     a = exp(-c softplus(decay_d) sigma(r))       v = sqrt(1 - a^2) sigma(i) x
    log       a = exp(r)                                   v = x

Norms (``add_norm``, ``gated_norm`` and their backward passes), per row
    add_norm     s = residual + alpha scale_d x,  y = norm(s) w (+ b)
    gated_norm   n = norm(x SiLU(z)) w (+ b)      or  n = (norm(x) w (+ b)) SiLU(z)
                 out = n                          or  out = residual + alpha scale_d n
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
CKPT = 64       # the forward keeps the state entering every 64th step for the backward
EPS = 1e-6
GATE_SCALE = 8.0


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # decoding for a few users: one token each through the recurrence
        dict(name="step_few", op="step", gate="decay", z=True, dtype="bf16", batch=4, d=1536),
        # decoding for many users at the large width
        dict(name="step_many", op="step", gate="sigmoid", z=True, dtype="f32", batch=256, d=5120),
        # a few prompts of odd length and width, state kept for decoding
        dict(name="scan_prompt", op="scan", gate="log", z=False, dtype="f16", batch=3, seq_len=517, d=1001,
             reset=False, h0=True),
        # one long document read at once: few channels, many steps
        dict(name="scan_long", op="scan", gate="decay", z=True, dtype="bf16", batch=1, seq_len=65536, d=2560,
             reset=False, h0=False),
        # a training step on packed documents: forward, then all gradients
        dict(name="scan_train_packed", op="scan_train", gate="decay", z=False, dtype="bf16", batch=8, seq_len=2048,
             d=1536, reset=True, h0=False),
        # a training step at the large width, gated output
        dict(name="scan_train_large", op="scan_train", gate="sigmoid", z=True, dtype="f32", batch=4, seq_len=8192,
             d=5120, reset=False, h0=True),
        # the norm before a block while decoding: a handful of rows
        dict(name="add_norm_tokens", op="add_norm", kind="rms", dtype="bf16", res="f32", rows=16, d=2560,
             scale=False, bias=False),
        # the norm before a block in training, residual stream in 32 bits, a learned residual scale
        dict(name="add_norm_train", op="add_norm_train", kind="rms", dtype="bf16", res="f32", rows=32768, d=2560,
             scale=True, bias=False),
        # the same with a mean and a bias at an odd width and a ragged number of rows
        dict(name="add_norm_train_odd", op="add_norm_train", kind="layer", dtype="f16", res="f16", rows=1551, d=1001,
             scale=False, bias=True),
        # the gated norm of eight groups of channels after a scan, on a prompt
        dict(name="gated_norm_prompt", op="gated_norm", kind="rms", order="before", dtype="bf16", rows=1999, d=5120,
             groups=8, residual=False, bias=False),
        # the gated norm in training
        dict(name="gated_norm_train", op="gated_norm_train", kind="rms", order="before", dtype="bf16", rows=32768,
             d=5120, groups=1, residual=False, bias=False),
        # the norm that closes a block: gate after the norm, scaled into the residual
        dict(name="gated_norm_train_residual", op="gated_norm_train", kind="layer", order="after", dtype="f32",
             rows=16384, d=768, groups=1, residual=True, bias=True),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["step", "scan", "scan", "scan_train", "scan_train", "add_norm", "add_norm_train", "gated_norm",
                     "gated_norm_train"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    d = _log_int(rng, 32, 5120)
    if rng.random() < 0.5:
        d = max(8, d // 8 * 8)
    if op == "step":
        return dict(op=op, gate=rng.choice(["sigmoid", "decay", "log"]), z=rng.random() < 0.5, dtype=dtype,
                    batch=_log_int(rng, 1, 256), d=d)
    if op in ("scan", "scan_train"):
        batch = _log_int(rng, 1, 8)
        most = min(65536, (1 << 26) // (batch * d))
        return dict(op=op, gate=rng.choice(["sigmoid", "decay", "log"]), z=rng.random() < 0.5, dtype=dtype,
                    batch=batch, seq_len=_log_int(rng, 16, most), d=d, reset=rng.random() < 0.4,
                    h0=rng.random() < 0.5)
    rows = _log_int(rng, 1, min(32768, (1 << 26) // d))
    kind = rng.choice(["rms", "layer"])
    if op in ("add_norm", "add_norm_train"):
        return dict(op=op, kind=kind, dtype=dtype, res=rng.choice(["f32", dtype]), rows=rows, d=d,
                    scale=rng.random() < 0.5, bias=rng.random() < 0.5)
    groups = rng.choice([g for g in (1, 2, 4, 8) if d % g == 0])
    return dict(op=op, kind=kind, order=rng.choice(["before", "after"]), dtype=dtype, rows=rows, d=d, groups=groups,
                residual=rng.random() < 0.5, bias=rng.random() < 0.5)


# ----------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    t = DTYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0, dtype=t):
        x = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=g)
        return x.to(dtype)

    d, s = case["d"], dict(case=dict(case))
    f32 = torch.float32
    if case["op"] in ("step", "scan", "scan_train"):
        batch, seq_len = case["batch"], case.get("seq_len", 1)
        rows = batch * seq_len
        s["x"] = normal(rows, d)
        # gates as projections give them: most states kept for tens of steps
        if case["gate"] == "log":
            s["r"] = (-torch.exp(normal(rows, d, std=1.0, mean=-2.5, dtype=f32))).to(t)
        else:
            s["r"] = normal(rows, d, mean=2.0 if case["gate"] == "sigmoid" else 0.0)
        decay = case["gate"] == "decay"
        s["i"] = normal(rows, d) if decay else None
        # softplus(decay) such that a ** (1 / sigma) lies in 0.9 .. 0.999
        lam = torch.empty(d, device="cuda").uniform_(0.9, 0.999, generator=g)
        s["decay"] = torch.log(torch.expm1(-torch.log(lam) / GATE_SCALE)) if decay else None
        s["z"] = normal(rows, d) if case["z"] else None
        if case["op"] == "step":
            s["h"] = normal(batch, d, dtype=f32)
            return s
        s["h0"] = normal(batch, d, dtype=f32) if case["h0"] else None
        s["reset"] = None
        if case["reset"]:
            # packed documents, about eight a row, one starting each row
            u = torch.empty(batch, seq_len, device="cuda").uniform_(0, 1, generator=g)
            u[:, 0] = 0
            s["reset"] = (u < 8.0 / seq_len).to(torch.uint8).reshape(rows)
        if case["op"] == "scan_train":
            s["dout"] = normal(rows, d)
            s["dh_last"] = normal(batch, d, dtype=f32) if case["h0"] else None
        return s
    rows = case["rows"]
    s["x"] = normal(rows, d)
    s["weight"] = normal(d, std=0.2, mean=1.0, dtype=f32)
    s["bias"] = normal(d, std=0.2, dtype=f32) if case["bias"] else None
    if case["op"].startswith("add_norm"):
        s["residual"] = normal(rows, d, std=2.0, dtype=DTYPES[case["res"]])
        s["scale"] = normal(d, std=0.2, mean=1.0, dtype=f32) if case["scale"] else None
        s["alpha"] = 0.7
        if case["op"].endswith("train"):
            s["dy"] = normal(rows, d)
            s["ds"] = normal(rows, d, dtype=DTYPES[case["res"]])
        return s
    s["z"] = normal(rows, d)
    s["residual"] = normal(rows, d, std=2.0) if case["residual"] else None
    s["scale"] = normal(d, std=0.2, mean=1.0, dtype=f32) if case["residual"] else None
    s["alpha"] = 0.7 if case["residual"] else 1.0
    if case["op"].endswith("train"):
        s["dout"] = normal(rows, d)
    return s


# --------------------------------------------------------------- the one pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import mamba_selective_scan_causal_amd as mss
    c = s["case"]
    op = c["op"]
    if op == "step":
        y = mss.gated_step(s["x"], s["r"], s["i"], s["decay"], s["z"], s["h"], gate=c["gate"],
                           gate_scale=GATE_SCALE)
        return dict(y=y, h=s["h"])
    if op in ("scan", "scan_train"):
        train = op == "scan_train"
        size = dict(batch=c["batch"], seq_len=c["seq_len"], gate=c["gate"], gate_scale=GATE_SCALE)
        y, ckpt, h_last = mss.gated_scan(s["x"], s["r"], s["i"], s["decay"], s["z"], s["h0"], s["reset"],
                                         h_ckpt=train, h_last=True, **size)
        if not train:
            return dict(y=y, h_last=h_last)
        grads = mss.gated_scan_backward(s["x"], s["r"], s["i"], s["decay"], s["z"], s["reset"], ckpt, s["dout"],
                                        dh_last=s["dh_last"], need_dh0=c["h0"], **size)
        return dict(grads, y=y, h_last=h_last)
    kind = dict(kind=c["kind"], eps=EPS, alpha=s["alpha"])
    if op.startswith("add_norm"):
        y, r = mss.add_norm(s["x"], s["residual"], s["weight"], s["bias"], s["scale"], **kind)
        if op == "add_norm":
            return dict(y=y, residual=r)
        grads = mss.add_norm_backward(r, s["weight"], s["dy"], s["ds"], s["x"], s["scale"],
                                      bias=s["bias"] is not None, **kind)
        return dict(grads, y=y, residual=r)
    more = dict(kind, groups=c["groups"], order=c["order"])
    y = mss.gated_norm(s["x"], s["z"], s["weight"], s["bias"], s["residual"], s["scale"], **more)
    if op == "gated_norm":
        return dict(y=y)
    grads = mss.gated_norm_backward(s["x"], s["z"], s["weight"], s["bias"], s["scale"], s["dout"], **more)
    return dict(grads, y=y)


# ------------------------------------------------------------ the plain forms

def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _silu_and_slope(v):
    s = _sigmoid(v)
    return v * s, s * (1.0 + v * (1.0 - s))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _scan(a, b):
    """h_t = b_t + a_t h_{t-1} from h = 0 along dim 1, in log2(L) doublings."""
    step = 1
    while step < a.shape[1]:
        tail = a[:, step:].clone()
        b = torch.cat([b[:, :step], b[:, step:] + tail * b[:, :-step]], 1)
        a = torch.cat([a[:, :step], tail * a[:, :-step]], 1)
        step *= 2
    return b


def _gates(c, x, r, i, decay):
    """(a, v, and what the backward pass needs of them) of every token."""
    if c["gate"] == "log":
        return torch.exp(r), x, ()
    s = _sigmoid(r)
    if c["gate"] == "sigmoid":
        keep = _sigmoid(-r)
        return s, keep * x, (keep,)
    k = GATE_SCALE * _softplus(decay)
    la = -k * s
    m = torch.sqrt(-torch.expm1(2.0 * la))
    g = _sigmoid(i)
    return torch.exp(la), m * g * x, (s, k, m, g)


def _plain(s):
    c = s["case"]
    op = c["op"]
    return (_plain_step if op == "step" else _plain_scan if op.startswith("scan") else
            _plain_add_norm if op.startswith("add_norm") else _plain_gated_norm)(s, c)


def _f(v):
    return None if v is None else v.float()


def _plain_step(s, c):
    a, v, _ = _gates(c, _f(s["x"]), _f(s["r"]), _f(s["i"]), s["decay"])
    s["h"].copy_(v + a * s["h"])
    y = s["h"] if s["z"] is None else s["h"] * _silu_and_slope(_f(s["z"]))[0]
    return dict(y=y.to(s["x"].dtype), h=s["h"])


def _plain_scan(s, c):
    shape, t = (c["batch"], c["seq_len"], c["d"]), s["x"].dtype
    x, r, i, z = (None if s[k] is None else s[k].float().reshape(shape) for k in ("x", "r", "i", "z"))
    a, v, more = _gates(c, x, r, i, s["decay"])
    carry = a if s["reset"] is None else a * (s["reset"].reshape(*shape[:2], 1) == 0)
    if s["h0"] is not None:
        v = torch.cat([v[:, :1] + (carry[:, 0] * s["h0"])[:, None], v[:, 1:]], 1)
    h = _scan(carry, v)
    gate, slope = _silu_and_slope(z) if z is not None else (None, None)
    y = (h if z is None else h * gate).to(t).reshape(s["x"].shape)
    out = dict(y=y, h_last=h[:, -1].clone())
    if c["op"] == "scan":
        return out
    dout = s["dout"].float().reshape(shape)
    dy = dout if z is None else dout * gate
    if s["dh_last"] is not None:
        dy = torch.cat([dy[:, :-1], (dy[:, -1] + s["dh_last"])[:, None]], 1)
    zero = torch.zeros_like(h[:, :1])
    grad = _scan(torch.cat([zero, carry[:, 1:].flip(1)], 1), dy.flip(1)).flip(1)
    first = zero if s["h0"] is None else s["h0"][:, None]
    before = torch.cat([first, h[:, :-1]], 1)
    if s["reset"] is not None:
        before = before * (s["reset"].reshape(*shape[:2], 1) == 0)
    di = ddecay = None
    if c["gate"] == "log":
        dx, dr = grad, grad * a * before
    elif c["gate"] == "sigmoid":
        keep, = more
        dx, dr = grad * keep, grad * (before - x) * a * keep
    else:
        sig, k, m, g = more
        dx, di = grad * m * g, grad * m * x * g * (1.0 - g)
        w = grad * (a * before - x * g * a * a / m)
        dr = -w * k * sig * (1.0 - sig)
        ddecay = (-(w * sig).double().sum((0, 1)) * GATE_SCALE * _sigmoid(s["decay"].double())).float()
    flat = lambda v: None if v is None else v.to(t).reshape(s["x"].shape)  # noqa: E731
    return dict(out, dx=flat(dx), dr=flat(dr), di=flat(di), ddecay=ddecay,
                dz=None if z is None else flat(dout * h * slope),
                dh0=carry[:, 0] * grad[:, 0] if c["h0"] else None)


def _normed(v, kind):
    """(normalised v, 1 / its deviation) over the last dim."""
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    rstd = 1.0 / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)
    return v * rstd, rstd


def _normed_backward(g, n, rstd, kind):
    """Gradient of what was normalised to n, for a gradient g of n."""
    d = g - n * (g * n).mean(-1, keepdim=True)
    return (d - g.mean(-1, keepdim=True) if kind == "layer" else d) * rstd


def _rows_sum(v):
    return v.double().sum(0).float()


def _plain_add_norm(s, c):
    x, t = s["x"].float(), s["x"].dtype
    k = s["alpha"] if s["scale"] is None else s["alpha"] * s["scale"]
    res = (s["residual"].float() + k * x).to(s["residual"].dtype)
    n, rstd = _normed(res.float(), c["kind"])
    y = n * s["weight"]
    y = (y if s["bias"] is None else y + s["bias"]).to(t)
    if c["op"] == "add_norm":
        return dict(y=y, residual=res)
    dy = s["dy"].float()
    dres = s["ds"].float() + _normed_backward(dy * s["weight"], n, rstd, c["kind"])
    return dict(y=y, residual=res, dx=(k * dres).to(t), dresidual=dres.to(s["residual"].dtype),
                dweight=_rows_sum(dy * n), dbias=None if s["bias"] is None else _rows_sum(dy),
                dscale=None if s["scale"] is None else s["alpha"] * _rows_sum(dres * x))


def _plain_gated_norm(s, c):
    shape, t = s["x"].shape, s["x"].dtype
    x, z = s["x"].float(), s["z"].float()
    gate, slope = _silu_and_slope(z)
    before = c["order"] == "before"
    split = lambda v: v.reshape(shape[0], c["groups"], -1)  # noqa: E731
    n, rstd = _normed(split(x * gate if before else x), c["kind"])
    n = n.reshape(shape)
    p = n * s["weight"]
    p = p if s["bias"] is None else p + s["bias"]
    q = p if before else p * gate
    k = s["alpha"] if s["scale"] is None else s["alpha"] * s["scale"]
    y = k * q if s["residual"] is None else s["residual"].float() + k * q
    if c["op"] == "gated_norm":
        return dict(y=y.to(t))
    dout = s["dout"].float()
    dq = k * dout
    dp = dq if before else dq * gate
    dv = _normed_backward(split(dp * s["weight"]), split(n), rstd, c["kind"]).reshape(shape)
    return dict(y=y.to(t), dx=(dv * gate if before else dv).to(t),
                dz=(dv * x * slope if before else dq * p * slope).to(t), dweight=_rows_sum(dp * n),
                dbias=None if s["bias"] is None else _rows_sum(dp),
                dscale=None if s["scale"] is None else s["alpha"] * _rows_sum(dout * q))


# --------------------------------------------------- what a pass cannot do without

def work(case):
    e, d = SIZE[case["dtype"]], case["d"]
    op = case["op"]
    if op in ("step", "scan", "scan_train"):
        n = case["batch"] * case.get("seq_len", 1) * d
        ins = 2 + (case["gate"] == "decay") + case["z"]          # x, r, i, z
        state = 4 * case["batch"] * d
        flops = {"sigmoid": 8, "decay": 20, "log": 4}[case["gate"]] + 6 * case["z"]
        if op == "step":
            return {"bytes": n * e * (ins + 1) + 2 * state, "flops": n * flops}
        rows = case["batch"] * case["seq_len"]
        if op == "scan":
            return {"bytes": n * e * (ins + 1) + state * (1 + case["h0"]) + rows * case["reset"], "flops": n * flops}
        # a step's outputs reach the loss between the two directions, so both read their inputs
        kept = 4 * case["batch"] * d * -(-case["seq_len"] // CKPT)
        return {"bytes": n * e * (ins + 1) + n * e * (2 * ins + 1) + 2 * kept + state * (1 + 3 * case["h0"])
                + 2 * rows * case["reset"], "flops": n * 4 * flops}
    n = case["rows"] * d
    if op.startswith("add_norm"):
        er = SIZE[case["res"]]
        forward = n * (2 * e + 2 * er)
        if op == "add_norm":
            return {"bytes": forward, "flops": n * 7}
        return {"bytes": forward + n * (2 * e + 3 * er + e * case["scale"]), "flops": n * 25}
    forward = n * e * (3 + case["residual"])
    if op == "gated_norm":
        return {"bytes": forward, "flops": n * 14}
    return {"bytes": forward + n * e * 5, "flops": n * 45}


# ------------------------------------------------------------ the exact values

def exact(case, seed):
    """The definition in 64 bits: the recurrence step by step in time, the norms by their moments; gradients by
    the chain rule of those steps (the recurrence) and by differentiating the definition (the norms)."""
    s = prepare(case, seed)
    return _exact_scan(s, case) if case["op"] in ("step", "scan", "scan_train") else _exact_norm(s, case)


def _exact_scan(s, c):
    batch, seq_len = c["batch"], c.get("seq_len", 1)
    time = lambda k: None if s.get(k) is None else s[k].double().reshape(batch, seq_len, -1).transpose(0, 1).contiguous()  # noqa: E731
    x, r, i, z, dout = (time(k) for k in ("x", "r", "i", "z", "dout"))
    decay = None if s["decay"] is None else s["decay"].double()
    if c["gate"] == "log":
        a, v = r.exp(), x
    elif c["gate"] == "sigmoid":
        a = torch.sigmoid(r)
        v = torch.sigmoid(-r) * x
    else:
        la = -GATE_SCALE * torch.nn.functional.softplus(decay) * torch.sigmoid(r)
        a, m = la.exp(), (-torch.expm1(2 * la)).sqrt()
        v = m * torch.sigmoid(i) * x
    step = c["op"] == "step"
    keep = torch.ones(seq_len, batch, 1, dtype=torch.float64, device=x.device)
    if s.get("reset") is not None:
        keep = (s["reset"].reshape(batch, seq_len).t() == 0).double()[..., None]
    start = s["h"] if step else s["h0"]
    start = torch.zeros_like(x[0]) if start is None else start.double()
    ak = a * keep
    h = torch.empty_like(x)
    now = start
    for t in range(seq_len):
        now = torch.addcmul(v[t], ak[t], now, out=h[t])
    y = h if z is None else h * z * torch.sigmoid(z)
    rows = lambda w: None if w is None else w.transpose(0, 1).reshape(batch * seq_len, -1)  # noqa: E731
    if step:
        return dict(y=rows(y), h=h[0])
    out = dict(y=rows(y), h_last=h[-1])
    if c["op"] == "scan":
        return out
    dh = dout.clone() if z is None else dout * z * torch.sigmoid(z)
    if s["dh_last"] is not None:
        dh[-1] += s["dh_last"].double()
    for t in range(seq_len - 2, -1, -1):
        dh[t].addcmul_(ak[t + 1], dh[t + 1])
    prev = torch.cat([start[None], h[:-1]], 0) * keep
    di = ddecay = None
    if c["gate"] == "log":
        dx, dr = dh, dh * prev * a
    elif c["gate"] == "sigmoid":
        dx, dr = dh * torch.sigmoid(-r), dh * (prev - x) * a * torch.sigmoid(-r)
    else:
        gi, sr = torch.sigmoid(i), torch.sigmoid(r)
        dx, di = dh * m * gi, dh * m * x * gi * torch.sigmoid(-i)
        da = dh * prev - dh * x * gi * a / m
        dr = da * a * -GATE_SCALE * torch.nn.functional.softplus(decay) * sr * torch.sigmoid(-r)
        ddecay = (da * a * -GATE_SCALE * sr).sum((0, 1)) * torch.sigmoid(decay)
    dz = None
    if z is not None:
        dz = dout * h * (torch.sigmoid(z) + z * torch.sigmoid(z) * torch.sigmoid(-z))
    return dict(out, dx=rows(dx), dr=rows(dr), di=rows(di), ddecay=ddecay, dz=rows(dz),
                dh0=ak[0] * dh[0] if c["h0"] else None)


def _exact_norm(s, c):
    train = c["op"].endswith("train")
    part, got = 8192, []
    for r0 in range(0, c["rows"], part):
        got.append(_exact_rows(s, c, train, slice(r0, min(c["rows"], r0 + part))))
    out = {}
    for k in got[0]:
        vs = [g[k] for g in got]
        out[k] = None if vs[0] is None else sum(vs) if k in ("dweight", "dbias", "dscale") else torch.cat(vs, 0)
    return out


def _exact_rows(s, c, train, cut):
    row = lambda k: None if s.get(k) is None else s[k][cut].double().requires_grad_(train and k not in ("dy", "ds", "dout"))  # noqa: E731
    par = lambda k: None if s.get(k) is None else s[k].double().requires_grad_(train)  # noqa: E731
    x, z, residual = row("x"), row("z"), row("residual")
    w, b, scale = par("weight"), par("bias"), par("scale")
    add = c["op"].startswith("add_norm")
    with torch.set_grad_enabled(train):
        k = s["alpha"] * (scale if scale is not None else 1.0)
        u = residual + k * x if add else x * torch.nn.functional.silu(z) if c["order"] == "before" else x
        # the norm reads the residual stream as its type holds it
        v = u + (u.to(s["residual"].dtype).double() - u).detach() if add else u.reshape(u.shape[0], c["groups"], -1)
        mu = v.mean(-1, keepdim=True) if c["kind"] == "layer" else 0.0
        var = ((v - mu) ** 2).mean(-1, keepdim=True)
        y = ((v - mu) * (var + EPS) ** -0.5).reshape(u.shape) * w + (b if b is not None else 0.0)
        if not add:
            y = y if c["order"] == "before" else y * torch.nn.functional.silu(z)
            y = k * y + (residual if residual is not None else 0.0)
    out = dict(y=y.detach())
    if add:
        out["residual"] = u.detach()
    if not train:
        return out
    if add:
        torch.autograd.backward([y, u], [s["dy"][cut].double(), s["ds"][cut].double()])
        out["dresidual"] = residual.grad
    else:
        y.backward(s["dout"][cut].double())
        out["dz"] = z.grad
    out["dx"], out["dweight"] = x.grad, w.grad
    out["dbias"] = None if b is None else b.grad
    out["dscale"] = None if scale is None else scale.grad
    return out
