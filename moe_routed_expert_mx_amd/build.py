"""Build the HIP library for gfx950 (hipcc) and the native binding of its dense side (g++), in-tree; no JIT cache.

The binding only makes calls shorter: where it cannot be built (no g++, no headers of Python or PyTorch), the build
says so, removes one that an older source left, and the package does without.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = [os.path.join(HERE, "csrc", name) for name in ("moe_mx.hip", "moe_dense.hip", "moe_norm.hip", "moe_f8.hip")]
LIB = os.path.join(HERE, "libmoe_mx.so")
BINDING_SOURCE = os.path.join(HERE, "csrc", "dense_binding.cpp")
BINDING = os.path.join(HERE, "_dense.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # packed FP32 instructions stay off: ordinary float code only
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def _run(cmd, verbose: bool) -> None:
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "packed-fp32-ops"
    msgs = "\n".join(ln for ln in (res.stdout + res.stderr).splitlines() if noise not in ln)
    if res.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed ({res.returncode}):\n{msgs}")
    if verbose and msgs.strip():
        print(msgs)


def build_library(verbose: bool = False) -> str:
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as d:
        objs = [os.path.join(d, os.path.basename(src) + ".o") for src in SOURCES]
        with ThreadPoolExecutor(len(SOURCES)) as pool:
            list(pool.map(lambda so: _run([HIPCC, *FLAGS, "-I", os.path.join(ROOT, "include"), "-c", so[0], "-o",
                                           so[1]], verbose), zip(SOURCES, objs)))
        _run([HIPCC, "--offload-arch=gfx950", "-shared", *objs, "-o", tmp], verbose)
    os.replace(tmp, LIB)
    return LIB


def build_binding(verbose: bool = False) -> str:
    """Host code only: it reads tensors through torch's headers and calls the library by address."""
    import torch
    from torch.utils.cpp_extension import include_paths
    tmp, libs = BINDING + ".tmp", os.path.join(os.path.dirname(torch.__file__), "lib")
    includes = [*include_paths(), sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-isystem{i}" for i in includes),
          BINDING_SOURCE, "-o", tmp, f"-L{libs}", f"-Wl,-rpath,{libs}", "-ltorch_python", "-ltorch", "-ltorch_cpu",
          "-lc10"], verbose)
    os.replace(tmp, BINDING)
    return BINDING


def build(verbose: bool = False) -> str:
    with ThreadPoolExecutor(2) as pool:
        binding = pool.submit(build_binding, verbose)
        lib = build_library(verbose)
        try:
            binding.result()
        except Exception as e:
            if os.path.exists(BINDING):
                os.remove(BINDING)
            print(f"native binding not built, calls of the dense side will take longer: {e}", file=sys.stderr)
    return lib


if __name__ == "__main__":
    print(build(verbose=True))
