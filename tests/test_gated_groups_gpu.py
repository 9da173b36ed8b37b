"""The gated recurrence over several groups of chunks, in each way that a launch
hands states over: groups of 32 chunks (at most 12 tiles of 64 fp32 or 128
2-byte channels), groups of 8, and groups of 8 with the tiles in eight sets."""
from __future__ import annotations

import pytest

from gpu_util import announce
from test_gated_gpu import run_case
from test_block_run_gpu import scan_both, scan_case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _announce(request):
    announce(request.node.nodeid)
    yield


# chunks are 128 steps forward, 64 backward
@pytest.mark.parametrize("B,L,D,dtype,gate", [
    (1, 9000, 130, "f32", "decay"),         # 3 tiles, groups of 32: 3 forward, 5 backward
    (3, 4500, 256, "f32", "log"),           # 12 tiles, the last with groups of 32
    (1, 3300, 832, "f32", "sigmoid"),       # 13 tiles, groups of 8: 4 and 7
    (1, 2049, 1664, "bf16", "decay"),       # 13 tiles of 2-byte channels, one step past a group
    (4, 1300, 512, "f32", "decay"),         # 32 tiles: 2 and 3 groups
    (2, 1025, 1000, "f16", "log"),          # 16 tiles, a ragged last one
    (8, 1100, 512, "f32", "sigmoid"),       # 64 tiles: sets
    (8, 1100, 1024, "bf16", "decay"),       # 64 tiles of 2-byte channels: sets
    (16, 700, 333, "f32", "log"),           # 96 tiles in sets, rows that start inside a line
    (2, 1200, 2049, "f32", "decay")])       # 66 tiles: no equal eighths
def test_several_groups(B, L, D, dtype, gate):
    run_case(B, L, D, gate, dtype, z=L % 2 == 0, h0=B % 2 == 0, reset=D % 2 == 0, decay_mean=-6.0)


@pytest.mark.parametrize("B,L,D,dtype", [(4, 1300, 512, "f32"), (8, 1100, 1024, "bf16"), (1, 9000, 130, "f32")])
def test_repeats_are_bit_identical(B, L, D, dtype):
    import torch
    g, k = scan_case(31, B, L, D, dtype)
    want = scan_both(g, k)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(scan_both(g, k), want))


def test_several_groups_in_a_graph():
    """Replays, with the eager calls on the same inputs and other work between them."""
    import torch
    cases = [scan_case(32, 8, 1100, 512, "f32"), scan_case(33, 4, 1300, 512, "f32", "sigmoid")]
    want = [t for g, k in cases for t in scan_both(g, k)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [t for g, k in cases for t in scan_both(g, k)]
    for _ in range(3):
        for t in got:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        scan_both(*cases[0])


def test_two_streams_over_groups_at_once():
    import torch
    cases = [scan_case(34, 8, 1100, 1024), scan_case(35, 1, 3300, 832, "f32")]
    want = [scan_both(g, k) for g, k in cases]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(4):
        for s, (g, k) in zip(streams, cases):
            got.append(scan_both(g, k, stream=s))
    torch.cuda.synchronize()
    for j, outs in enumerate(got):
        assert all(torch.equal(p, q) for p, q in zip(outs, want[j % 2]))
