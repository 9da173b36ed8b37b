"""A launch that fails is reported by the call that made it, whichever of its
launches it is, and nothing is launched after it.  The runtime's launch call is
replaced by one that runs nothing (launch_fails.cpp), so the pointers are fake
and no GPU is needed."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
EHIP = -5


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    lib = str(tmp_path_factory.mktemp("launch") / "liblaunch_fails.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-o", lib, os.path.join(HERE, "launch_fails.cpp")],
                   check=True, timeout=120)
    return lib


def calls():
    """(what, a function making the call, launches it needs)."""
    import test_block_abi_cpu as abi
    L = abi.mss.lib()
    for gate in (0, 1, 2):
        for steps in (60, 100, 300):
            over = {} if gate == 1 else dict(i=None, decay=None)
            back = over if gate == 1 else dict(over, di=None, ddecay=None)
            d = abi.gated(L=steps, gate=gate)
            # the marking of the workspace where there are several chunks (of 128 steps, of 64
            # in the backward), the scan, and the sum of ddecay
            yield (f"gated_scan gate {gate} L {steps}", lambda d=d, o=over: abi.call(L, "mss_gated_scan", d, **o),
                   1 + (steps > 128))
            yield (f"gated_scan_backward gate {gate} L {steps}",
                   lambda d=d, o=back: abi.call(L, "mss_gated_scan_backward", d, **o), 1 + (steps > 64) + (gate == 1))
    yield "gated_scan L 0", lambda: abi.call(L, "mss_gated_scan", abi.gated(L=0), ws_size=0), 1
    yield ("gated_scan_backward L 0",
           lambda: abi.call(L, "mss_gated_scan_backward", abi.gated(L=0), ws_size=0), 2)
    for name in abi.CALLS:
        if "gated_scan" in name:
            continue
        for width in ((64, 20000) if "norm" in name else (64,)):
            d = abi.norm(D=width) if "norm" in name else abi.gated()
            yield f"{name} D {width}", lambda d=d, n=name: abi.call(L, n, d), 2 if "norm_back" in name else 1


def child():
    control = ctypes.CDLL(os.environ["LAUNCH_FAILS"])
    for what, call, launches in calls():
        control.launch_fails_at(-1)
        status, seen = call(), control.launches_seen()
        assert (status, seen) == (0, launches), (what, status, seen)
        for n in range(launches):
            control.launch_fails_at(n)
            status, seen = call(), control.launches_seen()
            assert (status, seen) == (EHIP, n + 1), (what, f"launch {n} fails", status, seen)
    print("all reported")


def test_failed_launches_are_reported(stand_in):
    preload = os.pathsep.join(p for p in (stand_in, os.environ.get("LD_PRELOAD")) if p)
    env = dict(os.environ, LD_PRELOAD=preload, LAUNCH_FAILS=stand_in,
               PYTHONPATH=os.pathsep.join([HERE, os.path.dirname(HERE)]))
    r = subprocess.run([sys.executable, "-c", "import test_launch_errors_cpu as t; t.child()"], env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all reported" in r.stdout, (r.stdout + r.stderr)[-3000:]
