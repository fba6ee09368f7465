"""Build in-tree: liblora_linear.so with nvcc for sm_100a (B200), and _ops.so, the PyTorch side of the
operators around the layer (host code over that library)."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "liblora_linear.so")
OPS = os.path.join(HERE, "_ops.so")
SOURCES = [os.path.join(CSRC, f) for f in ("lora_linear.cu", "noalloc.cu", "merge.cu", "block.cu",
                                             "heads.cu", "decode.cu")]


def deps() -> list:
    """Every source the library is built from (all of csrc/ and the public header)."""
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))) + [
        os.path.join(ROOT, "include", "lora_linear.h"), os.path.abspath(__file__)]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
    "-Xptxas", "-O3",
    "--expt-relaxed-constexpr",
    "--threads", "4",  # the sources side by side
    "-shared",
]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or "/usr/local/cuda/bin/nvcc"
    return cand if os.path.exists(cand) else "nvcc"


def _older(target: str, sources) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in sources if os.path.exists(p))


def needs_build() -> bool:
    return _older(LIB, deps())


def build_ops(force: bool = False) -> str:
    """_ops.so, linked to liblora_linear.so beside it."""
    src, header = os.path.join(CSRC, "torch_ops.cpp"), os.path.join(ROOT, "include", "lora_linear.h")
    if not force and not _older(OPS, [src, header]):
        return OPS
    import torch
    base = os.path.dirname(torch.__file__)
    tmp = OPS + f".{os.getpid()}.tmp"
    inc = [os.path.join(ROOT, "include"), os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"]]
    # through nvcc, so that both libraries come from one host compiler
    cmd = [nvcc(), "-O2", "-std=c++17", "-shared", "--cudart", "none", "-Xcompiler", "-fPIC,-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-DTORCH_EXTENSION_NAME=_ops"]
    cmd += [f for d in inc for f in ("-isystem", d)] + ["-o", tmp, src, "-L", HERE, "-llora_linear", "-Xlinker",
                                                       "-rpath=$ORIGIN", "-L", os.path.join(base, "lib")]
    cmd += ["-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    subprocess.run(cmd, check=True)
    os.replace(tmp, OPS)
    return OPS


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        build_ops()
        return LIB
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [nvcc()] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-I", os.path.join(ROOT, "include"),
                                                                             "-o", tmp] + SOURCES
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    build_ops(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
