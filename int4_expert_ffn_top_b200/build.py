"""Build libmoe.so in-tree with nvcc for sm_100a, and the Python extension beside it with the host compiler and torch's
headers."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmoe.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_SOURCE = os.path.join(HERE, "csrc", "binding.cpp")
SOURCES = [os.path.join(HERE, "csrc", f) for f in ("moe_api.cu", "linear_api.cu")]
DEPS = [os.path.join(HERE, "csrc", f) for f in os.listdir(os.path.join(HERE, "csrc")) if f != "binding.cpp"] + [
    os.path.join(ROOT, "include", "moe.h")]

NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
              "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC", "-shared", "-Xptxas", "-O3"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def stale(target: str = LIB, deps: list[str] = DEPS) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def binding_tag() -> str:
    """What the extension says it was built for (``built_for``)."""
    import torch
    return f"moe binding for torch {torch.__version__}"


def binding_stale() -> bool:
    """Its sources are newer, or it was built for another torch."""
    if stale(BINDING, [BINDING_SOURCE, os.path.join(ROOT, "include", "moe.h")]):
        return True
    with open(BINDING, "rb") as f:
        return binding_tag().encode() + b"\0" not in f.read()


def binding_command(out: str) -> list[str]:
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.isabs(nvcc()) else "/usr/local/cuda"
    inc = [os.path.join(base, "include"), sysconfig.get_path("include"), os.path.join(cuda, "include")]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f'-DMOE_TORCH="{torch.__version__}"', f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-I{d}" for d in inc), "-o", out, BINDING_SOURCE, "-L" + os.path.join(base, "lib"), "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_python", "-ldl"]


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    if force or stale():
        cmd = [nvcc(), *NVCC_FLAGS, *(extra or []), "-o", LIB + ".tmp", *SOURCES]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
        os.replace(LIB + ".tmp", LIB)
    if force or binding_stale():
        cmd = binding_command(BINDING + ".tmp")
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.run(cmd, check=True)
        os.replace(BINDING + ".tmp", BINDING)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None)
