"""Build the HIP libraries ``libfp8q.so`` (the codec) and ``libfp8q_layer.so``
(the MoE layer's activation operators) in-tree for gfx950 with hipcc, and then
the Python module ``_layer.so`` over the second with g++ and torch's headers, a
step of its own: where those do not fit, the libraries are built all the same.

    python -m dequantize_reduce_transfer_amd.build

Cross-compiles without a GPU.  Flags:
  * ``--offload-arch=gfx950``  MI355X (CDNA4);
  * ``-ffp-contract=off``      every fp32 multiply and add is rounded on its
                               own, as the codec's definition requires (fused
                               multiply-adds are written out where intended);
  * ``-Xclang -target-feature -Xclang -packed-fp32-ops``  keeps the compiler
                               from forming packed fp32 instructions;
  * ``-mllvm -amdgpu-kernarg-preload-count=16``  the kernels' leading
                               arguments arrive preloaded in SGPRs instead of
                               through a scalar load at wave start (gfx950
                               supports it; the code object keeps a
                               fallback prologue); measured 0.5-1% faster for
                               the block quantize at 16-64 MiB payloads;
  * fp32 denormals stay enabled (no flush-to-zero flag).
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "libfp8q.so")
LAYER_LIB_PATH = os.path.join(PKG, "libfp8q_layer.so")
BINDING_PATH = os.path.join(PKG, "_layer.so")       # the Python module over libfp8q_layer.so

SOURCES = ["quantize.hip", "dequant_reduce.hip", "mx8_quantize.hip", "api.hip"]
LAYER_SOURCES = ["rms_norm.hip", "moe_sort.hip", "moe_rows.hip", "layer_api.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
CXXFLAGS = [
    "--offload-arch=" + ARCH, "-O3", "-fPIC", "-std=c++17", "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-mllvm", "-amdgpu-kernarg-preload-count=16",
    "-fvisibility=hidden", "-Wall", "-Wno-unused-function", "-I", INCLUDE, "-I", CSRC,
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *CXXFLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed on %s:\n%s\n%s" % (src, r.stdout, r.stderr))
    return obj


def _link(objs, lib: str) -> None:
    tmp = lib + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, lib)


def build_binding(verbose: bool = False) -> str:
    """Compile the Python module over libfp8q_layer.so (g++: host code only),
    which has to be built."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    tmp = BINDING_PATH + ".tmp%d" % os.getpid()
    lib = os.path.join(os.path.dirname(os.path.abspath(torch.__file__)), "lib")
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-I", INCLUDE,
           *["-isystem" + p for p in (*cpp_extension.include_paths(),
                                      sysconfig.get_paths()["include"])],
           os.path.join(CSRC, "layer_binding.cpp"), "-o", tmp, "-L", PKG, "-lfp8q_layer",
           "-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("building the layer binding failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, BINDING_PATH)
    if verbose:
        print("built", BINDING_PATH)
    return BINDING_PATH


def build(verbose: bool = False) -> str:
    """Compile every HIP source and link both libraries (always rebuilds); needs
    hipcc alone.  build_binding builds the Python module over the second."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    sources = [*SOURCES, *LAYER_SOURCES]
    with ThreadPoolExecutor(max_workers=min(len(sources), os.cpu_count() or 1)) as ex:
        objs = list(ex.map(_compile, sources))
    _link(objs[:len(SOURCES)], LIB_PATH)
    _link(objs[len(SOURCES):], LAYER_LIB_PATH)
    if verbose:
        print("built", LIB_PATH)
        print("built", LAYER_LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    build(verbose=True)
    build_binding(verbose=True)
    sys.exit(0)
