"""Build the HIP library ``libspa.so`` in-tree for gfx950 (hipcc, no JIT), and the native Python binding.

Usage: ``python -m activation_sparsification_amd.build`` (or call ``build()``).
Each ``csrc/*.hip`` is compiled to an object in ``_build/`` and the objects
are linked into ``activation_sparsification_amd/libspa.so``.
``native/layer_module.cpp`` (host code only, against torch's headers) becomes
``activation_sparsification_amd/_layer_native.so``, which loads the libspa.so
beside it.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libspa.so")
BINDING_SRC = os.path.join(PKG, "native", "layer_module.cpp")
BINDING = os.path.join(PKG, "_layer_native.so")
CXX = os.environ.get("CXX", "g++")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    "-Wno-unused-function",
    "-Wno-unused-command-line-argument",
    # packed fp32 instructions are kept out of the generated code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, *FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def _compile_binding() -> str:
    import torch
    tdir = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "layer_module.cpp.o")
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", os.path.join(ROOT, "include"),
           "-isystem", os.path.join(tdir, "include"), "-isystem", os.path.join(tdir, "include/torch/csrc/api/include"),
           "-isystem", os.path.join(ROCM, "include"), "-isystem", sysconfig.get_paths()["include"],
           "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{CXX} failed for {BINDING_SRC}:\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    tlib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    # torch's libraries are loaded by `import torch`, libspa.so is found beside the binding
    cmd = [CXX, "-shared", "-o", tmp, obj, "-L", PKG, "-l:libspa.so", "-Wl,-rpath,$ORIGIN", "-L", tlib, "-ltorch_python",
           "-ltorch_cpu", "-lc10_hip", "-lc10", "-Wl,--allow-shlib-undefined"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, srcs))
        binding = binding.result()
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding)
    if verbose:
        print(f"built {LIB} and {BINDING}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
