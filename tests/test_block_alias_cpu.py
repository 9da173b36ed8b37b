"""What may share memory in mss_add_norm updated in place, at the C ABI: the new
stream may be the residual, and nothing else."""
from __future__ import annotations

from test_block_abi_cpu import CALLS, EALIAS, L, call, fake, norm, strides  # noqa: F401 (L: fixture)

import mamba_selective_scan_causal_amd as mss

RES = CALLS["mss_add_norm"].index("residual") + 1


def test_x_may_not_be_the_stream_that_is_updated(L):  # noqa: F811
    """x, residual and s at one address: in one type, and as the halves of wider elements with
    rows that are equally far apart."""
    d = norm(M=4, D=64)
    assert call(L, "mss_add_norm", d, x=fake(RES), s=fake(RES)) == EALIAS
    st = strides(mss.NormStrides, 64)
    st.x = 128                                          # bf16 rows as far apart as fp32 ones
    d = norm(M=4, D=64, dtype=1, res=0)
    assert call(L, "mss_add_norm", d, st=st, x=fake(RES), s=fake(RES)) == EALIAS
    # the parameters neither
    d = norm(M=1, D=64, dtype=0, res=0)
    for name in ("w", "b", "scale"):
        assert call(L, "mss_add_norm", d, s=fake(RES), **{name: fake(RES)}) == EALIAS, name
