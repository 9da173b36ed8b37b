"""Every launch of the embedding, the head and clipping fails in turn: the call reports it and launches
nothing more.  As test_launch_errors_cpu.py does it for the block calls (the runtime's launch call is
replaced, no GPU is needed)."""
from __future__ import annotations

import ctypes
import os
import subprocess
import sys

from test_launch_errors_cpu import EHIP, HERE, stand_in  # noqa: F401


def calls():
    """(what, a function making the call)."""
    import test_ends_abi_cpu as abi
    L = abi.mss.lib()
    for M, V, D in ((10, 100, 64), (3000, 2000, 200), (10, 70000, 65), (0, 100, 64)):
        d = abi.embed(M, V, D)
        yield f"embedding_backward {M} {V} {D}", lambda d=d: abi.call(L, "mss_embedding_backward", d)
        if M:
            yield f"embedding {M}", lambda d=d: abi.call(L, "mss_embedding", d)
            yield f"accumulate {M}", lambda d=abi.embed(M, V, D, flags=1): abi.call(L, "mss_embedding_backward", d)
        for t in (0, 1, 2):
            h = abi.head(M, V, D, dtype=t)
            if M:
                yield f"head_loss {M} {V} {D} {t}", lambda h=h: abi.call(L, "mss_head_loss", h)
            yield f"head_loss_backward {M} {V} {D} {t}", lambda h=h: abi.call(L, "mss_head_loss_backward", h)
    # several pieces of the vocabulary, several groups of rows
    h = abi.head(40000, 70000, 64)
    yield "head_loss_backward in pieces", lambda: abi.call(L, "mss_head_loss_backward", h)
    yield "head_loss in groups", lambda: abi.call(L, "mss_head_loss", abi.head(1 << 20, 70000, 64))
    for count in (0, 1, 96, 97, 300):
        rows = [(abi.fake(0, 4096 * k), abi.fake(0, 4096 * k), 1000, k % 3, k % 3) for k in range(count)]
        for f in ("clip", "norm"):
            yield f"{f} of {count}", lambda rows=rows, f=f: abi.clip(L, rows, f=f)


def child():
    control = ctypes.CDLL(os.environ["LAUNCH_FAILS"])
    for what, call in calls():
        control.launch_fails_at(-1)
        status, launches = call(), control.launches_seen()
        assert status == 0 and 0 < launches < 100, (what, status, launches)
        for n in range(launches):
            control.launch_fails_at(n)
            status, seen = call(), control.launches_seen()
            assert (status, seen) == (EHIP, n + 1), (what, f"launch {n} fails", status, seen)
        print(what, launches)
    print("all reported")


def test_failed_launches_are_reported(stand_in):  # noqa: F811
    preload = os.pathsep.join(p for p in (stand_in, os.environ.get("LD_PRELOAD")) if p)
    env = dict(os.environ, LD_PRELOAD=preload, LAUNCH_FAILS=stand_in,
               PYTHONPATH=os.pathsep.join([HERE, os.path.dirname(HERE)]))
    r = subprocess.run([sys.executable, "-c", "import test_ends_launch_errors_cpu as t; t.child()"], env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all reported" in r.stdout, (r.stdout + r.stderr)[-3000:]
