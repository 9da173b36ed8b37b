"""Infinities in the norms' inputs: a channel that one lane reads for another
counts once, at every width."""
from __future__ import annotations

import numpy as np
import pytest

import mamba_selective_scan_causal_amd as mss
from block_util import back, put
from gpu_util import announce

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


# rows of whole vectors, and rows whose last vector reaches back over the one before
# (2-byte types: 8 channels), in teams of 16 and 64 lanes and of a workgroup
@pytest.mark.parametrize("D", (16, 13, 120, 125, 505, 1029, 2559))
@pytest.mark.parametrize("dtype", ("bf16", "f16", "f32"))
@pytest.mark.parametrize("which", ("x", "z"))
def test_an_infinite_channel_leaves_the_others_their_limit(D, dtype, which):
    """RMS with the gate before it: one infinite channel makes the norm infinite, so that the others
    are 0 w + b = b, and the channel itself inf / inf = NaN."""
    import torch
    rng = np.random.default_rng(D)
    M = D
    v = dict(x=rng.normal(size=(M, D)), z=rng.normal(size=(M, D)))
    at = rng.permutation(D)
    v[which][np.arange(M), at] = np.inf
    if which == "x":
        v["z"] = np.abs(v["z"]) + 0.1
    w, b = rng.normal(size=D), rng.normal(size=D)
    y = back(mss.gated_norm(put(v["x"], dtype), put(v["z"], dtype), put(w), put(b)))
    torch.cuda.synchronize()
    want = np.broadcast_to(back(put(back(put(b)), dtype)), (M, D)).copy()
    want[np.arange(M), at] = np.nan
    np.testing.assert_array_equal(y, want)


@pytest.mark.parametrize("D", (16, 13, 125, 1029))
@pytest.mark.parametrize("dtype", ("bf16", "f32"))
def test_an_infinite_residual_channel(D, dtype):
    import torch
    rng = np.random.default_rng(D)
    s, at = rng.normal(size=(D, D)), rng.permutation(D)
    s[np.arange(D), at] = -np.inf
    w, b = rng.normal(size=D), rng.normal(size=D)
    y, _ = mss.add_norm(put(rng.normal(size=(D, D)), dtype), put(s, dtype), put(w), put(b))
    torch.cuda.synchronize()
    want = np.broadcast_to(back(put(back(put(b)), dtype)), (D, D)).copy()
    want[np.arange(D), at] = np.nan
    np.testing.assert_array_equal(back(y), want)
