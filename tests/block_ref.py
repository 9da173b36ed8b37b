"""Plain fp64 forms of the gated recurrence and the block norms, step by step
from their definitions, with a bound on what fp32 evaluation may differ by.

The bounds count roundings: U = 2^-24 is half a step of fp32, and every
elementary function or operation on the way to a term is charged K U of the
term's absolute value (K = 64 covers the gates, whose exponentials lose up to
|r| U in their argument besides their own ulp, for |r| <= 40).  A recurrence
carries its error with the factor that it carries its state with, and the
absolute values are summed without cancellation, so the bounds hold for any
order in which the terms are combined.  An output of type T adds half a step
of T.

The decay gate's sigma(r), softplus(decay) and their product are 0 in fp32
where they lie below 2^-126, and its input scale m = sqrt(1 - a^2) <
sqrt(2 c softplus(decay) sigma(r)) is then 0 too: for c max(1, softplus) <= 32
that loses at most sqrt(64 2^-126) = UNDER of m, and of what m multiplies
(k sigma(r) / m < m as well, so dr's term over m is charged the same)."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
K = 64.0
UNDER = 2.0 ** -60
# half a step relative to the value, and half the smallest subnormal
HALF = {"f32": (U, 2.0 ** -126), "bf16": (2.0 ** -8, 2.0 ** -126), "f16": (2.0 ** -11, 2.0 ** -25)}


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def silu(v):
    return v * sigmoid(v)


def silu_slope(v):
    return sigmoid(v) * (1.0 + v * sigmoid(-v))


def tolerance(value, fp32_bound, dtype):
    rel, sub = HALF[dtype]
    # the rounded value is that of the fp32 result, not of the exact one
    return rel * (np.abs(value) + fp32_bound) + fp32_bound + sub


def gates(gate, x, r, i, k):
    """(a, v, and m, s, g of the decay gate)."""
    if gate == "sigmoid":
        return sigmoid(r), sigmoid(-r) * x, None
    if gate == "log":
        return np.exp(r), x, None
    s = sigmoid(r)
    la = -k * s
    m = np.sqrt(-np.expm1(2 * la))
    g = sigmoid(i)
    return np.exp(la), m * g * x, (m, s, g)


def gated_scan(x, r, i=None, decay=None, z=None, h0=None, reset=None, dout=None, dh_last=None, *,
               batch, seq_len, gate, gate_scale=8.0):
    """Values and bounds, each a dict of (M, D), (B, D) and (D,) arrays: y, h, h_last and, for
    a dout, dx, dr, di, dz, ddecay, dh0."""
    B, L, D = batch, seq_len, x.shape[1]
    tr = lambda v: None if v is None else np.asarray(v, np.float64).reshape(B, L, D)
    x, r, i, z, dout = (tr(v) for v in (x, r, i, z, dout))
    k = gate_scale * softplus(decay) if gate == "decay" else None
    with np.errstate(over="ignore"):
        a, v, more = gates(gate, x, r, i, k)
    keep = np.ones((B, L, 1)) if reset is None else (np.asarray(reset).reshape(B, L, 1) == 0) * 1.0
    under = UNDER * np.abs(x * more[2]) if gate == "decay" else np.zeros_like(x)
    start = np.zeros((B, D)) if h0 is None else np.asarray(h0, np.float64)
    h, ha, he = (np.empty((B, L, D)) for _ in range(3))
    p, pa, pe = (np.empty((B, L, D)) for _ in range(3))
    now, noa, noe = start, np.abs(start), np.zeros((B, D))
    for t in range(L):
        w = keep[:, t]
        p[:, t], pa[:, t], pe[:, t] = w * now, w * noa, w * noe
        now = a[:, t] * p[:, t] + v[:, t]
        noa = a[:, t] * pa[:, t] + np.abs(v[:, t])
        noe = a[:, t] * pe[:, t] + K * U * noa + under[:, t]
        h[:, t], ha[:, t], he[:, t] = now, noa, noe
    flat = lambda q: q.reshape(B * L, -1)
    f = 1.0 if z is None else silu(z)
    val = dict(y=flat(h * f), h=h, h_last=now)
    tol = dict(y=flat(np.abs(f) * (he + K * U * ha)), h=he, h_last=noe)
    if dout is None:
        return val, tol
    dy = dout * f
    G, Ga, Ge = (np.empty((B, L, D)) for _ in range(3))
    Q = np.zeros((B, D)) if dh_last is None else np.asarray(dh_last, np.float64)
    Qa, Qe = np.abs(Q), np.zeros((B, D))
    for t in range(L - 1, -1, -1):
        G[:, t] = dy[:, t] + Q
        Ga[:, t] = np.abs(dy[:, t]) + Qa
        Ge[:, t] = Qe + K * U * Ga[:, t]
        w = keep[:, t] * a[:, t]
        Q, Qa, Qe = w * G[:, t], w * Ga[:, t], w * (Ge[:, t] + K * U * Ga[:, t])
    val["dh0"], tol["dh0"] = Q, Qe

    def term(factor, other=None, other_abs=None, other_err=None):
        """G * factor * other with its bound; other = 1 when left out."""
        if other is None:
            return G * factor, np.abs(factor) * (Ge + K * U * Ga)
        return (G * factor * other,
                np.abs(factor) * (Ge * np.abs(other) + Ga * other_err + K * U * Ga * other_abs))

    if gate == "log":
        dx, ex = term(np.ones_like(a))
        dr, er = term(a, p, pa, pe)
    elif gate == "sigmoid":
        c = sigmoid(-r)
        dx, ex = term(c)
        dr, er = term(a * c, p - x, pa + np.abs(x), pe)
    else:
        m, s, g = more
        gc = sigmoid(-i)
        dx, ex = term(m * g)
        di, ei = term(m * g * gc * x)
        ex, ei = ex + UNDER * Ga * g, ei + Ga * under * gc
        val["di"], tol["di"] = flat(di), flat(ei)
        with np.errstate(invalid="ignore", divide="ignore"):
            q = np.where(m > 0, g * a * a * s / m, 0.0)
        ws, ew = term(np.ones_like(a), a * s * p - x * q, a * s * pa + np.abs(x) * q, a * s * pe)
        dr, er = -k * ws * sigmoid(-r), k * sigmoid(-r) * (ew + K * U * np.abs(ws)) + Ga * under
        scale = gate_scale * sigmoid(decay)
        val["ddecay"] = -scale * ws.sum((0, 1))
        # summed in fp32: at most 1024 + K roundings on the way of any term
        tol["ddecay"] = scale * (ew + (1024 + K) * U * np.abs(ws)).sum((0, 1))
    val["dx"], tol["dx"] = flat(dx), flat(ex)
    val["dr"], tol["dr"] = flat(dr), flat(er)
    if z is not None:
        slope = silu_slope(z)
        val["dz"] = flat(dout * h * slope)
        tol["dz"] = flat(np.abs(dout) * (he * np.abs(slope) + K * U * ha *
                                         (np.abs(slope) + sigmoid(z) * np.abs(z))))
    return val, tol


def moments(v, kind, eps):
    mean = v.mean(-1, keepdims=True) if kind == "layer" else np.zeros_like(v[..., :1])
    rstd = 1.0 / np.sqrt(((v - mean) ** 2).mean(-1, keepdims=True) + eps)
    # the mean is known to K U of the mean absolute value
    slack = np.abs(v).mean(-1, keepdims=True) * rstd if kind == "layer" else np.zeros_like(rstd)
    return (v - mean) * rstd, rstd, slack


def normed_backward(g, n, rstd, slack, kind):
    """Gradient of what was normalised to n for a gradient g of n, and its absolute terms."""
    c1, c2 = (g * n).mean(-1, keepdims=True), g.mean(-1, keepdims=True) * (kind == "layer")
    na = np.abs(n) + slack
    absolute = rstd * (np.abs(g) + na * (np.abs(g) * na).mean(-1, keepdims=True)
                       + np.abs(g).mean(-1, keepdims=True))
    return rstd * (g - n * c1 - c2), absolute


def add_norm(x, residual, scale, alpha):
    """(s before its rounding, its fp32 bound)."""
    k = alpha * (1.0 if scale is None else scale)
    base = 0.0 if residual is None else residual
    return base + k * x, 4 * U * (np.abs(base) + np.abs(k * x))


def norm_of(s, w, b, kind, eps):
    """norm(s) w + b and its fp32 bound."""
    n, _, slack = moments(s, kind, eps)
    b = 0.0 if b is None else b
    return n * w + b, K * U * ((np.abs(n) + slack) * np.abs(w) + np.abs(b))


def sums(v, extra=0.0):
    """Column sums and the bound of an fp32 sum of terms known to `extra`."""
    rows = v.shape[0]
    return v.sum(0), ((K + min(rows, 1024)) * U * np.abs(v) + extra).sum(0)


def add_norm_backward(s, w, dy, ds, x, scale, *, kind, eps, alpha):
    n, rstd, slack = moments(s, kind, eps)
    g = dy * w
    dv, dva = normed_backward(g, n, rstd, slack, kind)
    ds = np.zeros_like(s) if ds is None else ds
    dres, bound = ds + dv, 2 * K * U * (np.abs(ds) + dva)
    k = alpha * (1.0 if scale is None else scale)
    val, tol = dict(dresidual=dres, dx=k * dres), dict(dresidual=bound, dx=np.abs(k) * bound)
    val["dweight"], tol["dweight"] = sums(dy * n, K * U * np.abs(dy) * slack)
    val["dbias"], tol["dbias"] = sums(dy)
    if x is not None:
        val["dscale"], tol["dscale"] = sums(alpha * dres * x, np.abs(alpha * x) * bound)
    return val, tol


def gated_norm(x, z, w, b, residual, scale, dout=None, *, groups, order, kind, eps, alpha):
    M, D = x.shape
    split = lambda v: v.reshape(M, groups, D // groups)
    f, slope = (1.0, None) if z is None else (silu(z), silu_slope(z))
    before = order == "before"
    n, rstd, slack = moments(split(x * f if before else x), kind, eps)
    slack_c = np.broadcast_to(slack, n.shape).reshape(M, D)
    n_c = n.reshape(M, D)
    b = np.zeros(D) if b is None else b
    p, pa = n_c * w + b, (np.abs(n_c) + slack_c) * np.abs(w) + np.abs(b)
    q, qa = (p, pa) if before else (p * f, pa * np.abs(f))
    k = alpha * (np.ones(D) if scale is None else scale)
    base = np.zeros_like(x) if residual is None else residual
    val, tol = dict(y=base + k * q), dict(y=K * U * (np.abs(base) + np.abs(k) * qa))
    if dout is None:
        return val, tol
    dq = k * dout
    dp = dq if before else dq * f
    dv, dva = normed_backward(split(dp * w), n, rstd, slack, kind)
    dv, dva = dv.reshape(M, D), dva.reshape(M, D)
    fz = f if before else 1.0
    val["dx"], tol["dx"] = dv * fz, 2 * K * U * dva * np.abs(fz)
    if z is not None:
        slope_a = np.abs(slope) + sigmoid(z) * np.abs(z)
        val["dz"] = dv * x * slope if before else dq * p * slope
        tol["dz"] = 2 * K * U * (dva * np.abs(x) if before else np.abs(dq) * pa) * slope_a
    val["dweight"], tol["dweight"] = sums(dp * n_c, K * U * np.abs(dp) * slack_c)
    val["dbias"], tol["dbias"] = sums(dp)
    val["dscale"], tol["dscale"] = sums(alpha * dout * q, K * U * np.abs(alpha * dout) * qa)
    return val, tol
