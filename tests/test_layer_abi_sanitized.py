"""The layer operators' C-ABI layer under AddressSanitizer and
UndefinedBehaviorSanitizer, on the CPU: csrc/layer_api.hip compiled host-only
with g++, with tests/native/layer_stub_launchers.cpp in place of the kernels,
and every case of tests/test_layer_abi.py run against it in a child process,
the accepted calls included."""
import os
import re
import subprocess
import sys

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(ROOT, "dequantize_reduce_transfer_amd", "csrc")


def test_layer_abi_under_asan_ubsan(tmp_path):
    # libstdc++ too: the sanitizer looks for the function that throws when it
    # starts, and the binding's refusals are C++ exceptions
    runtimes = [subprocess.run(["gcc", "-print-file-name=" + n], capture_output=True, text=True).stdout.strip()
                for n in ("libasan.so", "libstdc++.so.6")]
    if not all(os.path.isabs(r) and os.path.exists(r) for r in runtimes):
        pytest.skip("sanitizer runtime not installed")
    lib = str(tmp_path / "libfp8q_layer_hostcheck.so")
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-Wall", "-D__HIP_PLATFORM_AMD__",
           "-I", os.path.join(rocm, "include"), "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer",
           "-fPIC", "-shared", "-o", lib,
           "-x", "c++", os.path.join(CSRC, "layer_api.hip"),
           "-x", "none", os.path.join(HERE, "native", "layer_stub_launchers.cpp")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ, FP8Q_LAYER_HOSTCHECK=lib, LD_PRELOAD=" ".join(runtimes), PYTHONMALLOC="malloc",
               ASAN_OPTIONS="detect_leaks=0:verify_asan_link_order=0:halt_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1:halt_on_error=1")
    r = subprocess.run([sys.executable, "-m", "pytest", os.path.join(HERE, "test_layer_abi.py"), "-q", "-s",
                        "-p", "no:cacheprovider", "-rs"], capture_output=True, text=True, timeout=600, env=env,
                       cwd=ROOT)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-4000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-4000:]
    assert re.search(r"(\d+) passed", out) and "skipped" not in out, out[-2000:]
