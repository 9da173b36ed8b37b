"""Rows whose loss weighs little beside another's: each row's dx has its own digits."""
from __future__ import annotations

import pytest
import torch

import ends_ref as ref
import mamba_selective_scan_causal_amd as mss
from ends_util import TYPES, check, spread
from gpu_util import announce
from test_head_gpu import case, run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


def check_rows(x, w, targets, dloss, dlse, got):
    """Each row's dx by the bound it has as a batch of its own; dweight by the batch's."""
    for m in range(x.shape[0]):
        one = slice(m, m + 1)
        want = ref.head(x[one], w, targets[one], 1.0, dloss[one], None if dlse is None else dlse[one])["dx"]
        check(got["dx"][one], want, f"dx of row {m}, dloss {dloss[m].item():.3g}")
    value, bound = ref.head(x, w, targets, 1.0, dloss, dlse)["dweight"]
    # sums past the type's largest number are infinite
    beyond = value.abs() + bound > torch.finfo(x.dtype).max
    here = got["dweight"].double().cpu()
    assert beyond.sum() < 0.01 * value.numel() and (here[beyond].abs() >= (value.abs() - bound)[beyond]).all()
    check(torch.where(beyond, value, here), (value, bound), "dweight")


@pytest.mark.parametrize("with_dlse", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,V,D", [(33, 3001, 64), (20, 9001, 71), (300, 2003, 40)])
def test_rows_of_any_weight(dtype, M, V, D, with_dlse):
    """Down to 2^-30 of the largest: fp16's numbers span 2^-24 to 2^16."""
    x, w, targets, _, dlse = case(M, M, V, D, TYPES[dtype])
    dloss = 2.0 ** (13.3 - 31.0 * torch.arange(M) / M)
    dlse = dloss * dlse.sign() * 0.1 if with_dlse else None
    got = run(x, w, targets, dloss, dlse)
    check_rows(x, w, targets, dloss, dlse, got)
    again = run(spread(x)[0], spread(w)[0], targets, dloss, dlse)
    check_rows(x, w, targets, dloss, dlse, again)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_row_of_infinite_weight(dtype):
    """It leaves the other rows' dx as they are, whatever their size."""
    M, V, D = 40, 700, 56
    x, w, targets, dloss, _ = case(1, M, V, D, TYPES[dtype])
    targets = targets.clamp(0, V - 1)
    for size in (1e-4, 1e4):
        dloss = torch.full((M,), size)
        want = run(x, w, targets, dloss, None)["dx"]
        dloss[7] = float("inf")
        got = run(x, w, targets, dloss, None)["dx"]
        rest = torch.arange(M, device="cuda") != 7
        assert not torch.isfinite(got[7]).any()
        # the same values times another factor: rounded alike, to one step of dl and one of dx
        off = 4 * ref.HALF[TYPES[dtype]] * want[rest].double().norm(dim=1, keepdim=True)
        assert ((got[rest].double() - want[rest].double()).abs() <= off).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_many_rows_of_any_weight(dtype):
    """Over 16384 rows, and dx in fp32 partial sums: a few rows against batches of their own."""
    M, V, D, t = 17001, 4001, 40, TYPES[dtype]
    x, w, targets, _, _ = case(2, M, V, D, t)
    dloss = 2.0 ** (13.3 - 31.0 * torch.rand(M, generator=torch.Generator().manual_seed(1)))
    a = [v.cuda() for v in (x, w, targets, dloss)]
    _, lse = mss.head_loss(*a[:3])
    got = mss.head_loss_backward(*a[:3], lse, a[3])["dx"]
    for m in torch.arange(0, M, 397).tolist() + [M - 1]:
        one = slice(m, m + 1)
        check(got[one], ref.head(x[one], w, targets[one], 1.0, dloss[one])["dx"], f"dx of row {m}")
