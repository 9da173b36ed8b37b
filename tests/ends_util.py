"""Comparisons and inputs shared by the tests of the embedding, the head's loss and clipping."""
from __future__ import annotations

import torch

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def generator(seed):
    return torch.Generator().manual_seed(seed)


def check(got, want, what):
    """|got - value| within the bound, everywhere; non-finite where and as the value is."""
    value, bound = want
    got = got.detach().double().cpu()
    assert got.shape == value.shape, (what, got.shape, value.shape)
    if value.numel() == 0:
        return 0.0
    err = (got - value).abs()
    bad = ~(err <= bound)
    worst = float((err / bound.clamp(min=1e-300)).masked_fill(bad, 0).max())
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at "
                           f"{tuple(torch.nonzero(bad)[0].tolist())}: got {got[bad][0].item()!r}, want "
                           f"{value[bad][0].item()!r}, bound {bound[bad][0].item():.3g}")
    return worst


def some_ids(g, M, V, dtype=torch.int64, away=0.1, crowd=0.3):
    """Ids with padding, ids past the table, one token in many places and the ends of the table."""
    ids = torch.randint(0, V, (M,), generator=g)
    u = torch.rand(M, generator=g)
    ids = torch.where(u < crowd, torch.full_like(ids, V // 3), ids)
    ids = torch.where(u > 1 - away, torch.full_like(ids, -100), ids)
    ids = torch.where((u > 1 - away) & (u < 1 - 2 * away / 3), torch.full_like(ids, V), ids)
    if M > 2:
        ids[0], ids[1] = 0, V - 1
    return ids.to(dtype)


def spread(t, extra=3, offset=1, fill=float("nan")):
    """The same values as a column range of a wider buffer: (view, buffer)."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    wide[:, offset:offset + t.shape[1]] = t
    return wide[:, offset:offset + t.shape[1]], wide
