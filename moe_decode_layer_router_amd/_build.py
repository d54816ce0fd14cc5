"""Build ``libmoeblk.so`` (all HIP sources, gfx950 only) in-tree with hipcc, and the
binding's argument check (``_marshal``, host code) with g++."""

from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmoeblk.so")
MARSHAL = os.path.join(PKG, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))  # of this Python alone
ARCH = "gfx950"

# -packed-fp32-ops: keep hipcc from emitting v_pk_{add,mul,fma}_f32 (hipcc's
# host pass warns that it does not know the feature; that is harmless).
HIPCC_FLAGS = [
    "-O3",
    "-std=c++17",
    f"--offload-arch={ARCH}",
    "-fPIC",
    "-shared",
    "-Wall",
    "-Wno-unused-function",
    "-Xclang",
    "-target-feature",
    "-Xclang",
    "-packed-fp32-ops",
]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def build_library(verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    tmp = LIB + ".tmp"
    cmd = [hipcc, *HIPCC_FLAGS, *(extra_flags or []), f"-I{INCLUDE}", f"-I{CSRC}", *sources(), "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
    if verbose and err.strip():
        print(err)
    os.replace(tmp, LIB)
    return LIB


def build_marshal(verbose: bool = False) -> str | None:
    """The check in C, for the Python and torch that build it. None, with a message, where that
    fails (no g++, or no headers): the binding then checks in Python, and finds no older file."""
    for old in (MARSHAL, os.path.join(PKG, "_marshal.so")):  # the latter: of any Python
        if os.path.exists(old):
            os.remove(old)
    tmp = MARSHAL + ".tmp"
    try:
        import torch
        from torch.utils import cpp_extension

        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall"]
        cmd += [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
        cmd += [f'-DMARSHAL_TORCH="{torch.__version__} {torch.version.git_version}"']
        cmd += [f"-isystem{i}" for i in (*cpp_extension.include_paths(), sysconfig.get_paths()["include"])]
        cmd += [os.path.join(CSRC, "marshal.cpp"), "-o", tmp]
        cmd += [f"-L{p}" for p in cpp_extension.library_paths()] + ["-ltorch_python", "-ltorch_cpu", "-lc10"]
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        error = f"{cmd[0]} failed ({res.returncode})\n{res.stderr}" if res.returncode != 0 else ""
    except (ImportError, OSError) as e:
        error = str(e)
    if error:
        print(f"the binding's check in C is not built, the one in Python serves:\n{error}", file=sys.stderr)
        return None
    if verbose and res.stderr.strip():
        print(res.stderr)
    os.replace(tmp, MARSHAL)
    return MARSHAL


if __name__ == "__main__":
    print(build_library(verbose=True))
    print(build_marshal(verbose=True))
