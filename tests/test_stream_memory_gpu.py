"""Calls on a stream that is not the current one, and the memory they allocate:
neither stream's work writes what the other still uses, also where results are
dropped at once or the memory was freed just before the call."""
from __future__ import annotations

import math

import pytest

import mamba_selective_scan_causal_amd as mss
from gpu_util import announce
from test_block_run_gpu import norm_both, norm_case, scan_both, scan_case

pytestmark = pytest.mark.gpu

BUSY = 20_000_000          # cycles of the spin kernel: about 10 ms


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


def block_calls():
    import torch
    g, k = scan_case(21, 2, 1500, 192)
    n = norm_case(22, 400, 640)

    def step(**more):
        return [mss.gated_step(g["x"][:2], g["r"][:2], g["i"][:2], g["decay"], g["z"][:2], g["h0"], gate="decay",
                               **more)]

    B, L, H, P, N = 2, 300, 8, 16, 16
    D, M = H * P, B * L

    def f(*shape):
        return torch.linspace(-1, 1, math.prod(shape), device="cuda").reshape(shape)

    p = {k: f(*shape) for k, shape in dict(x=(M, D), dt=(M, H), A=(D, N), A_h=(H,), B=(M, N), w=(D, 4), v=(D,),
                                           conv=(B, 3, D), h=(B, D, N)).items()}

    def core(**more):
        """The calls of the selective core, without its step."""
        kw = dict(batch=B, seq_len=L, **more)
        x, scan = p["x"], (p["x"], p["x"], p["A"], p["B"], p["B"])
        y, ck, hl = mss.selective_scan(*scan, disc="zoh", h_cache=True, h_last=True, ckpt8=True, **kw)
        y2, _, _ = mss.mamba1_core(x, p["w"], p["v"], *scan[1:], disc="zoh", **kw)
        g = mss.selective_scan_backward(*scan, p["v"], x, None, x, disc="zoh", need_dh0=True, **kw)
        g2 = mss.selective_scan_backward_noalloc(*scan, None, None, None, x, disc="zoh", **kw)
        ssd, state = mss.ssd_scan(x, p["dt"], p["A_h"], p["B"], p["B"], head_dim=P, d_state=N, disc="zoh",
                                  h_last=True, **kw)
        return [mss.conv1d_silu(x, p["w"], p["v"], **kw), y, ck, hl, y2, ssd, state,
                *mss.conv1d_silu_backward(x, p["w"], p["v"], x, **kw),
                *(v for d in (g, g2) for v in d.values() if v is not None)]

    def core_step(**more):
        return [mss.selective_step(p["x"][:B], None, p["x"][:B], p["A"], p["B"][:B], p["B"][:B], None, p["w"], None,
                                   p["conv"], p["h"], disc="zoh", **more)]

    return {"core": core, "core_step": core_step, "step": step, "scan": lambda **m: scan_both(g, k, **m),
            "norms": lambda **m: norm_both(n, **m)}


@pytest.mark.parametrize("what", ("scan", "norms", "step", "core", "core_step"))
def test_dropped_results_are_not_overwriting_the_current_streams(what):
    """The call waits on its stream; its results are dropped, and tensors of their sizes filled on
    the current stream.  What the call writes later must not land in them."""
    import torch
    call = block_calls()[what]
    sizes = [(t.shape, t.dtype) for t in call()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(s):
            torch.cuda._sleep(BUSY)
        call(stream=s)
        mine = [torch.full(shape, 7.0, dtype=t, device="cuda") for shape, t in sizes for _ in range(2)]
        torch.cuda.synchronize()
        assert all(bool((t == 7).all()) for t in mine)
        del mine


@pytest.mark.parametrize("what", ("scan", "norms", "step", "core", "core_step"))
def test_results_do_not_take_memory_that_the_current_stream_still_reads(what):
    """Tensors that the current stream has yet to read are dropped just before the call: its
    results, of their sizes, must not be written into them early."""
    import torch
    call = block_calls()[what]
    sizes = [(t.shape, t.dtype) for t in call()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        mine = [torch.full(shape, 7.0, dtype=t, device="cuda") for shape, t in sizes]
        torch.cuda.synchronize()
        torch.cuda._sleep(BUSY)
        copies = [t.clone() for t in mine]
        del mine
        got = call(stream=s)
        torch.cuda.synchronize()
        assert all(bool((t == 7).all()) for t in copies)
        del got, copies


@pytest.mark.parametrize("what", ("scan", "norms", "core"))
def test_results_used_on_the_current_stream_afterwards(what):
    """Results used on the current stream and dropped while that use is still to come, with more
    calls on the stream behind them: the use sees the results."""
    import torch
    call = block_calls()[what]
    want = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = call(stream=s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(BUSY)
        copies = [t.clone() for t in got]
        del got
        with torch.cuda.stream(s):
            junk = [torch.full_like(t, 7.0) for t in want]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(copies, want))
        del junk, copies


def test_a_captured_call_on_a_side_stream():
    """A graph whose calls run on a stream that forks from the captured one, some results dropped
    inside: every replay gives the eager bits."""
    import torch
    calls = block_calls()
    want = calls["scan"]() + calls["norms"]()
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        calls["scan"](stream=s)
        got = calls["scan"](stream=s) + calls["norms"](stream=s)
        torch.cuda.current_stream().wait_stream(s)
    for _ in range(3):
        for t in got:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        calls["scan"](stream=s)
        torch.cuda.synchronize()
