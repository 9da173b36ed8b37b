"""Parameter blocks and sizes that the binding keeps: values, never objects of
the caller's, and never an object that the caller holds."""
from __future__ import annotations

import pytest

import mamba_selective_scan_causal_amd as mss


@pytest.mark.parametrize("make,field", [(lambda: mss.make_gated_dims(2, 3, 4, 0, 1), "batch"),
                                        (lambda: mss.make_norm_dims(5, 8, 0, 0, 0), "rows"),
                                        (lambda: mss.make_gated_strides(4, 4), "x"),
                                        (lambda: mss.make_norm_strides(4, 4), "x")])
def test_a_block_is_the_callers_own(make, field):
    block = make()
    was = getattr(block, field)
    setattr(block, field, 77)
    assert getattr(make(), field) == was


class Recorder:
    """In the place of the library: keeps the parameter block that a call was given."""

    def __init__(self):
        self.blocks = []

    def __getattr__(self, name):
        def call(dims, *args):
            block = dims._obj
            if "workspace" in name:
                args[-1]._obj.value = int(block.batch * block.seq_len) if hasattr(block, "batch") else block.rows
                return 0
            self.blocks.append({k: getattr(block, k) for k, _ in block._fields_})
            return 0
        return call


@pytest.fixture
def recorded(monkeypatch):
    """The binding's calls on CPU tensors, with nothing behind them."""
    import torch
    r = Recorder()
    monkeypatch.setattr(mss, "lib", lambda: r)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)      # what CPU tensors report
    monkeypatch.setattr(torch.Tensor, "is_cuda", True)
    monkeypatch.setattr(mss._Call, "stream", lambda self: None)
    return r


def test_scalars_are_read_at_every_call(recorded):
    """A tensor given for a number is read when the call is made, not remembered by its identity."""
    import torch
    x, w = torch.zeros(6, 8), torch.ones(8)
    one = {k: torch.tensor(1.0, dtype=torch.float64) for k in ("alpha", "eps", "scale")}
    n = {k: torch.tensor(v) for k, v in dict(batch=2, seq_len=3, groups=2).items()}

    def calls():
        kw = dict(batch=n["batch"], seq_len=n["seq_len"], gate="decay", gate_scale=one["scale"])
        mss.gated_scan(x, x, x, w, **kw)
        mss.gated_scan_backward(x, x, x, w, None, None, torch.zeros(int(n["batch"]), 1, 8), x, **kw)
        mss.gated_step(x, x, x, w, None, x.clone(), gate="decay", gate_scale=one["scale"])
        kw = dict(alpha=one["alpha"], eps=one["eps"])
        mss.add_norm(x, x, w, **kw)
        mss.add_norm_backward(x, w, x, **kw)
        kw["groups"] = n["groups"]
        mss.gated_norm(x, x, w, **kw)
        mss.gated_norm_backward(x, x, w, None, None, x, **kw)

    calls()
    for v in one.values():
        v.mul_(2)
    n["batch"].fill_(3), n["seq_len"].fill_(2), n["groups"].fill_(4)
    calls()
    first, second = recorded.blocks[:7], recorded.blocks[7:]
    assert len(second) == 7
    for a, b in zip(first[:3], second[:3]):
        assert (a["gate_scale"], b["gate_scale"]) == (1.0, 2.0)
    for a, b in zip(first[:2], second[:2]):
        assert (a["batch"], a["seq_len"], b["batch"], b["seq_len"]) == (2, 3, 3, 2)
    for a, b in zip(first[3:], second[3:]):
        assert (a["alpha"], b["alpha"], a["eps"], b["eps"]) == (1.0, 2.0, 1.0, 2.0)
    for a, b in zip(first[5:], second[5:]):
        assert (a["groups"], b["groups"]) == (2, 4)


def test_sizes_are_read_at_every_query():
    import torch
    B = torch.tensor(2)
    ask = lambda: (mss.gated_workspace_bytes(mss.OP_GATED_SCAN_BACKWARD, batch=B, seq_len=700, d_inner=64, gate="log"),
                   mss.norm_workspace_bytes(mss.OP_ADD_NORM_BACKWARD, rows=B, width=64))
    small = ask()
    B.fill_(200)
    assert all(b > a for a, b in zip(small, ask()))
