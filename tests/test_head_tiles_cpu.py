"""The sizes that test_head_tiles_gpu.py runs launch every kernel of the head's products that the library
holds: each tile, layout and type.  The runtime's calls are replaced by ones that keep the kernels' names
(launch_names.cpp), so no GPU is needed."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


def products(names):
    return {n for n in names.decode().split() if any(f"head_{k}_kernel" in n for k in ("loss", "dl", "grad"))}


def child():
    names = ctypes.CDLL(os.environ["LAUNCH_NAMES"])
    names.kernels_held.restype = names.kernels_launched.restype = ctypes.c_char_p
    import test_ends_abi_cpu as abi
    from head_tiles import SIZES
    L = abi.mss.lib()
    held, reached = products(names.kernels_held()), set()
    assert held
    for dtype, M, V, D, strided in SIZES:
        dims = abi.head(M, V, D, dtype=("f32", "bf16", "f16").index(dtype))
        strides = abi.mss.make_head_strides(*[D + 3] * 4) if strided else None
        for call in ("mss_head_loss", "mss_head_loss_backward"):
            assert abi.call(L, call, dims, strides) == 0
        now = products(names.kernels_launched())
        print(dtype, M, V, D, strided, len(now))
        reached |= now
    missing = held - reached
    assert not missing, "\n".join(sorted(missing))
    print(f"all {len(held)} reached")


def test_every_tile_is_reached(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    lib = str(tmp_path / "liblaunch_names.so")
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-o", lib, os.path.join(HERE, "launch_names.cpp")],
                   check=True, timeout=120)
    preload = os.pathsep.join(p for p in (lib, os.environ.get("LD_PRELOAD")) if p)
    env = dict(os.environ, LD_PRELOAD=preload, LAUNCH_NAMES=lib,
               PYTHONPATH=os.pathsep.join([HERE, os.path.dirname(HERE)]))
    r = subprocess.run([sys.executable, "-c", "import test_head_tiles_cpu as t; t.child()"], env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "reached" in r.stdout, (r.stdout + r.stderr)[-5000:]
