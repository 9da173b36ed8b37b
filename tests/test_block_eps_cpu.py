"""The norms' eps at the C ABI: a normal fp32 number.  (v_rsq_f32 takes a
subnormal for 0, so that a row of zeros would come out NaN.)"""
from __future__ import annotations

import pytest

from test_block_abi_cpu import CALLS, EALIAS, EINVAL, OPS, L, norm, refused  # noqa: F401 (L: fixture)


@pytest.mark.parametrize("name", [n for n in CALLS if "norm" in n])
def test_subnormal_eps_is_refused(L, name):  # noqa: F811
    for eps in (1e-45, 1e-39, 1.17e-38):
        kw = dict(ws_size=1 << 40) if name in OPS else {}
        assert refused(L, name, norm(eps=eps), **kw) == EINVAL, eps
    assert refused(L, name, norm(eps=1.1754943508222875e-38)) == EALIAS       # 2^-126: valid but for the overlap
