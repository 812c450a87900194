"""Compile the library (HIP kernels for gfx950 + host code) into ``libentro.so``,
and the attention calls' binding to torch tensors into ``_attn.so``.

    python -m entropy_coded_weight_canonical_amd.build

Always rebuilds.  The shared objects land next to this file so that they ship
with the source tree.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libentro.so")
BINDING = os.path.join(HERE, "_attn.so")
SOURCES = ["entro_decode.hip", "entro_rans.hip", "entro_attn_prompt.hip", "entro_kv.hip", "entro_attn_cache.hip",
           "entro_lut.cpp", "entro_encode.cpp", "entro_rans.cpp"]
ARCH = os.environ.get("ENTRO_OFFLOAD_ARCH", "gfx950")


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def build(verbose: bool = False) -> str:
    objs = []
    common = ["-O3", "-std=c++17", "-fPIC", f"-I{INCLUDE}", f"-I{CSRC}", "-Wall", "-Wno-unused-function"]
    build_dir = os.path.join(HERE, "_build")
    os.makedirs(build_dir, exist_ok=True)
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(build_dir, src + ".o")
        if src.endswith(".hip"):
            cmd = [hipcc(), "-x", "hip", f"--offload-arch={ARCH}", "-munsafe-fp-atomics",
                   "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                   "-c", path, "-o", obj] + common
        else:
            rocm_inc = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")
            cmd = [hipcc(), "-x", "c++", f"-I{rocm_inc}", "-D__HIP_PLATFORM_AMD__", "-c", path, "-o", obj] + common
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)
        objs.append(obj)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs + ["-lpthread"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    build_binding(verbose)
    return LIB


def build_binding(verbose: bool = False) -> None:
    """``_attn.so`` (host code only; left out where torch is not installed)."""
    try:
        import torch
        from torch.utils.cpp_extension import include_paths
    except ImportError:
        return
    rocm_inc = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")
    includes = [INCLUDE, rocm_inc, sysconfig.get_paths()["include"]] + include_paths()
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + [f"-I{p}" for p in includes]
           + [os.path.join(CSRC, "entro_attn_py.cpp"), "-o", tmp,
              "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"])
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    os.replace(tmp, BINDING)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
