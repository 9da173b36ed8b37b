"""Each tile of the head's products, at the ends of its rows, its columns and its stages, against float64."""
from __future__ import annotations

import pytest
import torch

import ends_ref as ref
import mamba_selective_scan_causal_amd as mss
from ends_util import TYPES, check, spread
from gpu_util import announce
from head_tiles import SIZES
from test_head_extremes_gpu import INF, masked
from test_head_gpu import case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,M,V,D,strided", SIZES)
def test_tile(dtype, M, V, D, strided):
    announce(f"{dtype} {M} {V} {D} {strided}")
    x, w, targets, dloss, dlse = [v.cuda() for v in case(M + V, M, V, D, TYPES[dtype])]
    want = {k: [u.cpu() for u in v] for k, v in ref.head(x, w, targets, 1.0, dloss, dlse).items()}
    xs, ws = (spread(x)[0], spread(w)[0]) if strided else (x, w)
    loss, lse = mss.head_loss(xs, ws, targets)
    got = mss.head_loss_backward(xs, ws, targets, lse, dloss, dlse)
    torch.cuda.synchronize()
    for k, v in dict(got, loss=loss, lse=lse).items():
        announce(f"{k} {check(v, want[k], k):.2f} of the bound")


@pytest.mark.parametrize("infinite", [False, True])
@pytest.mark.parametrize("dtype,M,V,D,strided", SIZES)
def test_tile_with_masked_tokens_and_padded_rows(dtype, M, V, D, strided, infinite):
    """Several waves' tokens masked by the type's least value or by -inf, padded rows of NaN."""
    announce(f"{dtype} {M} {V} {D} {strided} {infinite}")
    v = torch.arange(V)
    off = ((v >= V // 3) & (v < V // 3 + 700)) | (v == V - 1)
    off[:2] = False
    value = -INF if infinite else torch.finfo(TYPES[dtype]).min
    x, w, keep, targets, dloss = masked(M + V, M, V, D, dtype, off, value)
    targets[1::5] = -100
    padded = targets < 0
    x[padded] = float("nan")
    xs, ws, t, d = [u.cuda() for u in (x, w, targets, dloss)]
    if strided:
        xs, ws = spread(xs)[0], spread(ws)[0]
    loss, lse = mss.head_loss(xs, ws, t)
    got = mss.head_loss_backward(xs, ws, t, lse, d)
    torch.cuda.synchronize()
    assert (got["dx"][padded.cuda()] == 0).all() and (loss[padded.cuda()] == 0).all()
    on, where = ~padded, torch.full((V,), -100)
    where[keep] = torch.arange(len(keep))
    want = ref.head(*[u.cuda() for u in (x[on], w[keep], where[targets[on]])], 1.0, d[on.cuda()])
    want = {k: [u.cpu() for u in p] for k, p in want.items()}
    at = on.cuda()
    check(loss[at], want["loss"], "loss")
    check(lse[at], want["lse"], "lse")
    columns = slice(1 if infinite else 0, None)          # 0 * -inf in the constant's own gradient
    check(got["dx"][at][:, columns], [u[:, columns] for u in want["dx"]], "dx")
    check(got["dweight"][keep.cuda()], want["dweight"], "dweight")
    assert (got["dweight"][off.cuda()] == 0).all()
