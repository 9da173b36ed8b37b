"""MSS_GATE_LOG with r > 0: states that grow.  The product of a chunk's factors
(128 steps at most) has to be finite, that of several chunks need not be."""
from __future__ import annotations

import numpy as np
import pytest

import block_ref as ref
import mamba_selective_scan_causal_amd as mss
from block_util import check, to_gpu
from gpu_util import announce

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


# 2 tiles (chunks in groups of 32, four to a wave) and 13 tiles (groups of 8)
@pytest.mark.parametrize("D", (70, 832))
@pytest.mark.parametrize("L", (500, 2700, 5000))
def test_products_past_the_range_of_fp32(L, D):
    """128 steps of e^0.5 make e^64, 256 of them no fp32 number.  The inputs are 0 but for the last
    120 steps (the gradients: but for the first 120), and a few tiny ones 300 steps off that end in
    some channels, which grow by e^100 and e^60 to values that fp32 holds."""
    import torch
    rng = np.random.default_rng(L + D)
    n = lambda *s: rng.normal(size=s)
    r, x, dout = np.full((L, D), 0.5), np.zeros((L, D)), np.zeros((L, D))
    x[-120:], dout[:120] = n(120, D), n(120, D)
    x[-300, ::3], dout[300, ::3] = 1e-37, 1e-37
    r[-200:-100], r[101:201] = 0.0, 0.0
    a = dict(x=x, r=r, i=None, decay=None, z=None, h0=None, reset=None, dout=dout, dh_last=None)
    g, e = to_gpu(a, "f32")
    kw = dict(batch=1, seq_len=L, gate="log")
    y, ck, hl = mss.gated_scan(g["x"], g["r"], h_ckpt=True, h_last=True, **kw)
    got = mss.gated_scan_backward(g["x"], g["r"], None, None, None, None, ck, g["dout"], need_dh0=True, **kw)
    torch.cuda.synchronize()
    val, tol = ref.gated_scan(**e, **kw)
    check(y, val["y"], tol["y"], "f32", "y")
    check(hl, val["h_last"], tol["h_last"], "f32", "h_last")
    for k in ("dx", "dr", "dh0"):
        check(got[k], val[k], tol[k], "f32", k)
