"""block_api.hip's host checks under AddressSanitizer and
UndefinedBehaviorSanitizer, as test_abi_sanitized.py does it for mss_api.hip:
compiled again with the sanitizers on its host code only, linked with the
regular objects, and driven through sizes and strides to the ends of int64."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

import mamba_selective_scan_causal_amd as mss
from mamba_selective_scan_causal_amd import build as hip_build

HERE = os.path.dirname(os.path.abspath(__file__))
SAN = "address,undefined"
CLANGXX = ("/opt/rocm/llvm/bin/clang++", "/opt/rocm/lib/llvm/bin/clang++")


@pytest.fixture(scope="module")
def sanitized_driver(tmp_path_factory):
    cxx = next((c for c in CLANGXX if os.path.exists(c)), None)
    if cxx is None or shutil.which(hip_build.hipcc()) is None:
        pytest.skip("hipcc / clang++ not available")
    mss.lib()
    rest = [os.path.join(hip_build.OBJDIR, s.replace(".hip", ".o")) for s in hip_build.SOURCES
            if s != "block_api.hip"]
    missing = [k for k in rest if not os.path.exists(k)]
    if missing:
        pytest.skip(f"objects missing: {missing}")
    out = tmp_path_factory.mktemp("asan_block")
    api_o, lib, exe = (str(out / n) for n in ("block_api_san.o", "libmss_block_san.so", "abi_block_sanitized"))
    hipcc = hip_build.hipcc()
    host_san = ["-Xarch_host", f"-fsanitize={SAN}", "-Xarch_host", "-fno-sanitize-recover=all",
                "-Xarch_host", "-fno-omit-frame-pointer", "-Xarch_host", "-g"]
    cmds = [
        [hipcc, *hip_build.FLAGS, *host_san, "-c", os.path.join(hip_build.CSRC, "block_api.hip"), "-o", api_o],
        [hipcc, f"--offload-arch={hip_build.ARCH}", "-shared", "-fPIC", "-Xarch_host",
         f"-fsanitize={SAN}", "-o", lib, api_o, *rest],
        [cxx, "-std=c++17", "-O1", "-g", f"-fsanitize={SAN}", "-fno-sanitize-recover=all",
         "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__", "-I", hip_build.INCLUDE,
         "-I", "/opt/rocm/include", os.path.join(HERE, "abi_block_sanitized.cpp"), lib,
         f"-Wl,-rpath,{out}", "-Wl,-rpath,/opt/rocm/lib", "-L/opt/rocm/lib", "-lamdhip64", "-o", exe],
    ]
    for c in cmds:
        r = subprocess.run(c, capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, " ".join(c) + "\n" + hip_build._quiet(r.stderr)[-3000:]
    return exe


def test_host_checks_clean_under_asan_ubsan(sanitized_driver):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1:abort_on_error=0",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sanitized_driver], capture_output=True, text=True, env=env, timeout=300)
    report = r.stdout + r.stderr
    assert r.returncode == 0 and "all checks passed" in r.stdout, report[-4000:]
    assert "runtime error" not in report and "AddressSanitizer" not in report, report[-4000:]
