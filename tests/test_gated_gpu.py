"""The gated linear recurrence on the GPU: forward, backward and single-token
step against the fp64 forms of block_ref, within their derived bounds."""
from __future__ import annotations

import numpy as np
import pytest

import block_ref as ref
import mamba_selective_scan_causal_amd as mss
from block_util import (back, check, column_slice, gated_inputs, outside_is_nan, put, to_gpu,
                        torch_type)
from gpu_util import announce

pytestmark = pytest.mark.gpu

GATES = ("sigmoid", "decay", "log")


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


def forward(g, kw, **more):
    return mss.gated_scan(g["x"], g["r"], g["i"], g["decay"], g["z"], g["h0"], g["reset"], **kw, **more)


def backward(g, kw, ck, dout, **more):
    return mss.gated_scan_backward(g["x"], g["r"], g["i"], g["decay"], g["z"], g["reset"], ck, dout,
                                   **kw, **more)


def run_case(B, L, D, gate, dtype, seed=0, dh_last=True, **opt):
    import torch
    rng = np.random.default_rng(1000 * seed + B + 10 * L + 7 * D)
    a = gated_inputs(rng, B, L, D, gate, **opt)
    a["dout"] = rng.normal(size=(B * L, D))
    a["dh_last"] = rng.normal(size=(B, D)) if dh_last else None
    g, e = to_gpu(a, dtype)
    kw = dict(batch=B, seq_len=L, gate=gate, gate_scale=8.0)
    y, ck, hl = forward(g, kw, h_ckpt=True, h_last=True)
    grads = backward(g, kw, ck, g["dout"], dh_last=g["dh_last"], need_dh0=True)
    torch.cuda.synchronize()
    val, tol = ref.gated_scan(**e, **kw)
    worst = {"y": check(y, val["y"], tol["y"], dtype, "y"),
             "h_last": check(hl, val["h_last"], tol["h_last"], "f32", "h_last")}
    enter = np.arange(0, L, mss.GATED_CKPT_STEPS)
    first = np.zeros((B, 1, D)) if e["h0"] is None else e["h0"][:, None]
    want = np.concatenate([first, val["h"]], 1)[:, enter]
    bound = np.concatenate([0 * first, tol["h"]], 1)[:, enter]
    worst["h_ckpt"] = check(ck, want, bound, "f32", "h_ckpt")
    for k, v in grads.items():
        if v is None:
            assert k not in val
            continue
        worst[k] = check(v, val[k], tol[k], dtype if k in ("dx", "dr", "di", "dz") else "f32", k)
    announce(f"B{B} L{L} D{D} {gate} {dtype} worst " + " ".join(f"{k}={v:.2f}" for k, v in worst.items()))


@pytest.mark.parametrize("dtype", ("f32", "bf16", "f16"))
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("z", (False, True))
def test_types_and_gates(dtype, gate, z):
    run_case(2, 333, 130, gate, dtype, z=z, h0=True, reset=True)


# lengths around the checkpoint spacing and the kernels' own block sizes; one
# channel, widths around a wave and its multiples, odd widths
@pytest.mark.parametrize("B,L,D", [(1, 1, 1), (3, 2, 5), (1, 63, 64), (2, 64, 63), (2, 65, 65), (1, 127, 128),
                                   (1, 128, 127), (2, 129, 129), (1, 255, 256), (1, 257, 100), (5, 17, 33),
                                   (1, 511, 2), (4, 513, 66), (1, 1024, 64), (1, 1025, 68), (7, 200, 72)])
@pytest.mark.parametrize("gate,dtype", [("decay", "bf16"), ("sigmoid", "f32")])
def test_sizes(B, L, D, gate, dtype):
    run_case(B, L, D, gate, dtype, z=(L + D) % 2 == 0, h0=D % 2 == 0, reset=L % 2 == 0, dh_last=B % 2 == 0)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_long_sequence_few_channels(gate, dtype):
    """Carries over many blocks: states that decay over hundreds of steps."""
    run_case(1, 5000, 34, gate, dtype, z=False, h0=True, decay_mean=-7.0)


@pytest.mark.parametrize("L", (1, 7, 8, 9, 15, 16, 17, 24, 31, 33, 47, 56, 57, 95, 113))
def test_many_short_sequences(L):
    """Workgroups of fewer waves, where one chunk holds the whole sequence."""
    run_case(9, L, 70, "decay", "bf16", z=L % 2 == 0, h0=True, reset=True, seed=L)


def test_many_rows():
    run_case(40, 70, 96, "sigmoid", "f16", z=True, h0=False)


def test_batch_and_width_past_one_wave_of_blocks():
    run_case(3, 300, 2000, "decay", "bf16", z=False, h0=False, reset=True)


# tiles of 64 (fp32) or 128 channels: counts around 64, multiples of eight and
# others, rows that start inside a cache line, where the tiles of a launch are
# kept together by eighths
@pytest.mark.parametrize("B,L,D,dtype", [(4, 300, 1000, "f32"), (4, 300, 1024, "f32"), (4, 150, 1473, "f32"),
                                         (1, 129, 4097, "f32"), (8, 40, 2303, "f32"), (8, 100, 2560, "f32"),
                                         (4, 300, 2047, "bf16"), (4, 300, 2048, "bf16"), (7, 140, 2045, "f16"),
                                         (7, 20, 2048, "bf16"), (8, 140, 2048, "bf16")])
def test_many_tiles(B, L, D, dtype):
    run_case(B, L, D, "sigmoid" if D % 2 else "decay", dtype, z=D % 3 == 0, h0=True, reset=L != 300)


@pytest.mark.parametrize("gate", GATES)
def test_every_step_reset(gate):
    """Nothing is ever carried: h = v, dh0 = 0, and what h0 holds does not matter."""
    import torch
    rng = np.random.default_rng(5)
    B, L, D = 2, 140, 40
    a = gated_inputs(rng, B, L, D, gate, z=False, h0=True)
    a["reset"] = np.full(B * L, 255, np.uint8)
    a["dout"] = rng.normal(size=(B * L, D))
    g, e = to_gpu(a, "f32")
    g["h0"].fill_(float("inf"))
    kw = dict(batch=B, seq_len=L, gate=gate)
    y, ck, hl = forward(g, kw, h_ckpt=True, h_last=True)
    grads = backward(g, kw, ck, g["dout"], need_dh0=True)
    torch.cuda.synchronize()
    val, tol = ref.gated_scan(**e, **kw)
    check(y, val["y"], tol["y"], "f32", "y")
    check(grads["dx"], val["dx"], tol["dx"], "f32", "dx")
    check(grads["dr"], val["dr"], tol["dr"], "f32", "dr")
    assert not grads["dh0"].any()


def test_reset_as_bool_and_packed_documents_equal_separate_ones():
    import torch
    rng = np.random.default_rng(6)
    lengths, D = [1, 70, 64, 129, 3], 50
    L = sum(lengths)
    a = gated_inputs(rng, 1, L, D, "decay", z=True, h0=False)
    g, e = to_gpu(a, "f32")
    starts = np.cumsum([0] + lengths[:-1])
    reset = torch.zeros(L, dtype=torch.bool, device="cuda")
    reset[torch.from_numpy(starts).cuda()] = True
    y, _, _ = mss.gated_scan(g["x"], g["r"], g["i"], g["decay"], g["z"], reset=reset, batch=1, seq_len=L,
                             gate="decay")
    for s, n in zip(starts, lengths):
        part = {k: e[k][s:s + n] for k in ("x", "r", "i", "z")}
        val, tol = ref.gated_scan(**part, decay=e["decay"], batch=1, seq_len=n, gate="decay")
        check(y[s:s + n], val["y"], tol["y"], "f32", f"document at {s}")


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("z", (False, True))
def test_nan_beyond_a_reset_stays_there(gate, z):
    """Documents of NaN and infinities (padding that nobody filled) before, between and after real
    ones, inside a piece of steps and across many chunks: the real ones' outputs and gradients are
    those of each alone."""
    import torch
    rng = np.random.default_rng(21)
    D, plan = 36, [(5, False), (3, True), (700, False), (130, True), (2, False), (64, False), (1, True), (9, False),
                   (300, False), (21, True)]                     # (length, real?)
    L = sum(n for n, _ in plan)
    a = gated_inputs(rng, 1, L, D, gate, z=z, h0=False)
    a["dout"] = rng.normal(size=(L, D))
    a["reset"] = np.zeros(L, np.uint8)
    starts = np.cumsum([0] + [n for n, _ in plan[:-1]])
    a["reset"][starts] = 1
    junk = np.concatenate([np.full(n, not real) for n, real in plan])
    for k in ("x", "r", "i", "z", "dout"):
        if a[k] is not None:
            a[k][junk] = rng.choice([np.nan, np.inf, -np.inf], size=(junk.sum(), D))
    for dtype in ("f32", "bf16"):
        g, e = to_gpu(a, dtype)
        kw = dict(batch=1, seq_len=L, gate=gate)
        y, ck, hl = forward(g, kw, h_ckpt=True, h_last=True)
        grads = backward(g, kw, ck, g["dout"])
        torch.cuda.synchronize()
        for s, (n, real) in zip(starts, plan):
            if not real:
                continue
            part = {k: None if e[k] is None else e[k][s:s + n] for k in ("x", "r", "i", "z", "dout")}
            val, tol = ref.gated_scan(**part, decay=e["decay"], batch=1, seq_len=n, gate=gate)
            check(y[s:s + n], val["y"], tol["y"], dtype, f"y of {n} at {s}")
            for k in ("dx", "dr", "di", "dz"):
                if grads[k] is not None:
                    check(grads[k][s:s + n], val[k], tol[k], dtype, f"{k} of {n} at {s}")
        check(hl, val["h_last"], tol["h_last"], "f32", "h_last")


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_closed_and_open_gates(gate, dtype):
    """r of -inf, very negative and very positive: the state is dropped, or kept untouched, and
    every gradient stays finite (the decay gate's, whose input scale has an infinite slope where
    it vanishes, takes its limit)."""
    import torch
    rng = np.random.default_rng(7)
    B, L, D = 1, 200, 24
    a = gated_inputs(rng, B, L, D, gate, z=False, h0=True)
    which = rng.integers(0, 5, size=(L, D))
    for n, v in enumerate((-np.inf, -200.0, -60.0)):
        a["r"][which == n] = v
    if gate == "sigmoid":
        a["r"][which == 3] = 60.0
    if gate == "decay":
        a["decay"][::3] = -30.0
        a["decay"][1::3] = -120.0
    a["dout"] = rng.normal(size=(L, D))
    g, e = to_gpu(a, dtype)
    kw = dict(batch=B, seq_len=L, gate=gate)
    y, ck, hl = forward(g, kw, h_ckpt=True, h_last=True)
    grads = backward(g, kw, ck, g["dout"], need_dh0=True)
    torch.cuda.synchronize()
    val, tol = ref.gated_scan(**e, **kw)
    check(y, val["y"], tol["y"], dtype, "y")
    for k, v in grads.items():
        if v is not None:
            assert torch.isfinite(v).all(), k
    check(grads["dx"], val["dx"], tol["dx"], dtype, "dx")
    check(grads["dr"], val["dr"], tol["dr"], dtype, "dr")


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("D", (96, 101))
def test_column_slices(dtype, D):
    """Every activation as a column range of a wider buffer, x and dx first: the values are the
    dense call's bit for bit and nothing outside the ranges is written."""
    import torch
    rng = np.random.default_rng(8)
    B, L = 2, 190
    a = gated_inputs(rng, B, L, D, "decay", z=True, h0=True, reset=True)
    a["dout"] = rng.normal(size=(B * L, D))
    g, _ = to_gpu(a, dtype)
    kw = dict(batch=B, seq_len=L, gate="decay")
    y, ck, hl = forward(g, kw, h_ckpt=True, h_last=True)
    grads = backward(g, kw, ck, g["dout"], need_dh0=True)
    s = dict(g)
    for n, k in enumerate(("x", "r", "i", "z", "dout")):
        s[k], _ = column_slice(g[k], extra=3 + n, offset=n % 3)
    out, wide = column_slice(torch.full_like(y, float("nan")))
    y2, ck2, hl2 = forward(s, kw, h_ckpt=True, h_last=True, out=out)
    places = {k: column_slice(torch.full_like(y, float("nan"))) for k in ("dx", "dr", "di", "dz")}
    grads2 = backward(s, kw, ck2, s["dout"], need_dh0=True, out={k: v[0] for k, v in places.items()})
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and torch.equal(hl2, hl) and torch.equal(ck2, ck)
    assert outside_is_nan(wide, D)
    for k, v in grads2.items():
        assert torch.equal(v, grads[k]), k
    for k, (_, w) in places.items():
        assert outside_is_nan(w, D), k


def test_gradients_side_by_side_in_one_buffer():
    """dx, dr, di, dz as neighbouring column ranges of one projection's gradient."""
    import torch
    rng = np.random.default_rng(9)
    B, L, D = 2, 100, 64
    a = gated_inputs(rng, B, L, D, "decay", z=True, h0=False)
    a["dout"] = rng.normal(size=(B * L, D))
    g, _ = to_gpu(a, "bf16")
    kw = dict(batch=B, seq_len=L, gate="decay")
    _, ck, _ = forward(g, kw, h_ckpt=True)
    want = backward(g, kw, ck, g["dout"])
    one = torch.full((B * L, 4 * D), float("nan"), dtype=torch.bfloat16, device="cuda")
    parts = dict(zip(("dx", "dr", "di", "dz"), one.split(D, 1)))
    backward(g, kw, ck, g["dout"], out=parts)
    torch.cuda.synchronize()
    for k, v in parts.items():
        assert torch.equal(v, want[k]), k


def test_empty():
    import torch
    f = dict(device="cuda")
    for B, L, D in ((0, 5, 8), (2, 5, 0)):
        x = torch.empty((B * L, D), **f)
        y, ck, hl = mss.gated_scan(x, x, batch=B, seq_len=L, gate="log", h_ckpt=True, h_last=True)
        assert y.shape == (B * L, D) and hl.shape == (B, D)
        mss.gated_scan_backward(x, x, None, None, None, None, ck, y, batch=B, seq_len=L, gate="log",
                                need_dh0=True)
        mss.gated_step(x[:B], x[:B], None, None, None, hl, gate="log") if D == 0 else None
    # no steps: the state passes through, both ways; nothing reaches decay
    x, h0 = torch.empty((0, 40), **f), torch.randn((2, 40), **f)
    kw = dict(batch=2, seq_len=0, gate="decay")
    dec = torch.zeros(40, **f)
    _, ck, hl = mss.gated_scan(x, x, x, dec, None, h0, h_ckpt=True, h_last=True, **kw)
    grads = mss.gated_scan_backward(x, x, x, dec, None, None, ck, x, dh_last=2 * h0, need_dh0=True, **kw)
    _, _, zero = mss.gated_scan(x, x, x, dec, h_last=True, **kw)
    torch.cuda.synchronize()
    assert torch.equal(hl, h0) and torch.equal(grads["dh0"], 2 * h0)
    assert not grads["ddecay"].any() and not zero.any()


@pytest.mark.parametrize("dtype", ("f32", "bf16", "f16"))
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("B,D", [(1, 1), (3, 65), (4, 1536), (64, 130)])
def test_step(dtype, gate, B, D):
    import torch
    rng = np.random.default_rng(B + D)
    a = gated_inputs(rng, B, 1, D, gate, z=B != 3, h0=True)
    g, e = to_gpu(a, dtype)
    h = g["h0"].clone()
    y = mss.gated_step(g["x"], g["r"], g["i"], g["decay"], g["z"], h, gate=gate)
    torch.cuda.synchronize()
    val, tol = ref.gated_scan(**e, batch=B, seq_len=1, gate=gate)
    check(y, val["y"], tol["y"], dtype, "y")
    check(h, val["h_last"], tol["h_last"], "f32", "h")


def test_steps_continue_a_scan():
    """A prompt through the scan, then tokens one by one with column-slice inputs: each equals
    the whole sequence's step."""
    import torch
    rng = np.random.default_rng(11)
    B, L, P, D = 3, 90, 70, 88
    a = gated_inputs(rng, B, L, D, "decay", z=True, h0=False)
    g, e = to_gpu(a, "bf16")
    val, tol = ref.gated_scan(**e, batch=B, seq_len=L, gate="decay")
    seq = lambda k: g[k].reshape(B, L, D)
    _, _, h = mss.gated_scan(*(seq(k)[:, :P].reshape(B * P, D) for k in ("x", "r", "i")), g["decay"],
                             seq("z")[:, :P].reshape(B * P, D), batch=B, seq_len=P, gate="decay", h_last=True)
    for t in range(P, L):
        both = torch.cat([seq("x")[:, t], seq("z")[:, t]], 1)
        y = mss.gated_step(both[:, :D], seq("r")[:, t], seq("i")[:, t], g["decay"], both[:, D:], h, gate="decay")
        check(y, val["y"].reshape(B, L, D)[:, t], tol["y"].reshape(B, L, D)[:, t], "bf16", f"y at {t}")
    check(h, val["h_last"], tol["h_last"], "f32", "h")


def test_left_padded_prompts():
    """Prompts of different lengths, padded on the left, with the reset on the first real token:
    final states as without the padding."""
    import torch
    rng = np.random.default_rng(12)
    lengths, L, D = [5, 140, 77], 140, 60
    a = gated_inputs(rng, 3, L, D, "sigmoid", z=False, h0=False)
    reset = np.zeros((3, L), np.uint8)
    for b, n in enumerate(lengths):
        reset[b, L - n] = 1
    a["reset"] = reset.reshape(-1)
    g, e = to_gpu(a, "f16")
    _, _, hl = forward(g, dict(batch=3, seq_len=L, gate="sigmoid"), h_last=True)
    torch.cuda.synchronize()
    for b, n in enumerate(lengths):
        cut = slice(b * L + L - n, (b + 1) * L)
        val, tol = ref.gated_scan(e["x"][cut], e["r"][cut], batch=1, seq_len=n, gate="sigmoid")
        check(hl[b:b + 1], val["h_last"], tol["h_last"], "f32", f"prompt {b}")


def test_repeats_are_bit_identical():
    import torch
    rng = np.random.default_rng(13)
    a = gated_inputs(rng, 2, 3000, 160, "decay", z=True, h0=True, reset=True)
    a["dout"] = rng.normal(size=(6000, 160))
    g, _ = to_gpu(a, "bf16")
    kw = dict(batch=2, seq_len=3000, gate="decay")
    first = None
    for _ in range(4):
        y, ck, hl = forward(g, kw, h_ckpt=True, h_last=True)
        grads = backward(g, kw, ck, g["dout"], need_dh0=True)
        got = [y, ck, hl, *(v for v in grads.values() if v is not None)]
        if first is None:
            first = got
        assert all(torch.equal(p, q) for p, q in zip(got, first))


def test_offsets_past_32_bits():
    """A buffer of more than 2^31 elements: x and y rows far apart; the last rows are right."""
    import torch
    L, D, ld = 9000, 4, 250000                       # 9000 * 250000 = 2.25e9 elements, bf16
    rng = np.random.default_rng(14)
    a = gated_inputs(rng, 1, L, D, "log", z=False, h0=False)
    g, e = to_gpu(a, "bf16")
    wide = torch.empty((L, ld), dtype=torch_type("bf16"), device="cuda")
    x, y = wide[:, :D], wide[:, D:2 * D]
    x.copy_(g["x"])
    mss.gated_scan(x, g["r"], batch=1, seq_len=L, gate="log", out=y)
    torch.cuda.synchronize()
    val, tol = ref.gated_scan(**e, batch=1, seq_len=L, gate="log")
    check(y.contiguous(), val["y"], tol["y"], "bf16", "y")


def test_binding_refuses():
    import torch
    f = dict(device="cuda")
    x = torch.zeros((12, 8), **f)
    kw = dict(batch=2, seq_len=6, gate="sigmoid")
    with pytest.raises(ValueError, match="gate must be"):
        mss.gated_scan(x, x, batch=2, seq_len=6, gate="tanh")
    with pytest.raises(ValueError, match="belong to gate='decay'"):
        mss.gated_scan(x, x, x, **kw)
    with pytest.raises(ValueError, match="i is required"):
        mss.gated_scan(x, x, batch=2, seq_len=6, gate="decay")
    with pytest.raises(TypeError, match="r must be"):
        mss.gated_scan(x, x.bfloat16(), **kw)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        mss.gated_scan(x.double(), x.double(), **kw)
    with pytest.raises(ValueError, match="expected shape"):
        mss.gated_scan(x, x[:6], **kw)
    with pytest.raises(ValueError, match="expected shape"):
        mss.gated_scan(x, x, reset=torch.zeros(11, dtype=torch.uint8, **f), **kw)
    with pytest.raises(ValueError, match="columns must be contiguous"):
        mss.gated_scan(x, torch.zeros((8, 12), **f).t(), **kw)
    with pytest.raises(ValueError, match="h_ckpt is required"):
        mss.gated_scan_backward(x, x, None, None, None, None, None, x, **kw)
    with pytest.raises(ValueError, match="no place"):
        mss.gated_scan_backward(x, x, None, None, None, None, torch.zeros((2, 1, 8), **f), x,
                                out={"dq": x}, **kw)
    with pytest.raises(mss.MssError) as err:
        mss.gated_scan(x, x, out=x, **kw)
    assert err.value.status == -3
    with pytest.raises(TypeError, match="reset must be"):
        mss.gated_scan(x, x, reset=[0] * 12, **kw)
    with pytest.raises(ValueError, match="on the GPU"):
        mss.gated_scan(x.cpu(), x, **kw)
    with pytest.raises(ValueError, match="current device"):
        mss.gated_scan(x, x.cpu(), **kw)
