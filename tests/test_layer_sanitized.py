"""The C ABI layer of the 8-bit layer around the dispatch (combine_moe_layout_02_amd/csrc/layer_api.cpp) compiled for the
host with g++ and the address and undefined-behaviour sanitizers, with launchers that only count calls, driven by
tests/c_abi/layer_asan.cpp. Runs on the CPU; no GPU code is built or run."""

import os
import shutil
import subprocess

import pytest

from conftest import ROOT

C_ABI = os.path.join(ROOT, "tests", "c_abi")
CSRC = os.path.join(ROOT, "combine_moe_layout_02_amd", "csrc")


def test_layer_calls_under_sanitizers(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists("/opt/rocm/include/hip/hip_runtime.h"):
        pytest.skip("needs g++ and the HIP headers")
    exe = tmp_path / "layer_asan"
    cmd = [gxx, "-std=c++17", "-g", "-O1", "-fno-omit-frame-pointer", "-fsanitize=address,undefined",
           "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}",
           os.path.join(CSRC, "layer_api.cpp"), os.path.join(C_ABI, "layer_asan.cpp"), "-o", str(exe)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0", UBSAN_OPTIONS="print_stacktrace=1")
    run = subprocess.run([str(exe)], capture_output=True, text=True, env=env, timeout=60)
    assert run.returncode == 0, run.stdout + run.stderr
    assert "layer_asan ok" in run.stdout
