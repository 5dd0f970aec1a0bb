"""Build libfa.so in-tree with nvcc for sm_100a.

    python -m exact_tiled_attention_36_b200.build

Compiles csrc/fa_api.cu (which includes the attention kernels' headers),
csrc/fa_noalloc.cu and csrc/fa_serve.cu (the 8-bit cache decode, the cache appends
and the block tables), side by side, and links them into
exact_tiled_attention_36_b200/libfa.so, with the CUDA runtime linked
statically so the library loads on a machine without a GPU driver (the
driver is reached at run time through the runtime's entry-point query). An object
whose source and headers did not change since it was built, by the same compiler and
flags, is used again, and so is the library; `extra` flags give objects of their own.
"""
from __future__ import annotations

import hashlib
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRCS = [os.path.join(HERE, "csrc", f) for f in ("fa_api.cu", "fa_noalloc.cu", "fa_serve.cu")]
OBJ_DIR = os.path.join(HERE, "_build")  # objects and their header lists
DEPS = [os.path.join(HERE, "csrc", f) for f in os.listdir(os.path.join(HERE, "csrc"))] + \
       [os.path.join(ROOT, "include", "fa.h")]
LIB = os.path.join(HERE, "libfa.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-std=c++17", "-O3", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC,-O2", "-cudart", "static",
    "--expt-relaxed-constexpr",
]


def _key(extra: list[str] | None) -> str:
    """Of the compiler and its flags: part of an object's name, and noted beside the library it went into."""
    return hashlib.sha256("\0".join([NVCC, *FLAGS, *(extra or [])]).encode()).hexdigest()[:12]


def _other_flags(key: str) -> bool:
    """Whether the library is noted to have been linked from objects of another key."""
    try:
        return open(os.path.join(OBJ_DIR, "linked")).read() != key
    except OSError:
        return False


def _fresh(obj: str) -> bool:
    """Whether `obj` is newer than every file its header list (make syntax) names, and this script."""
    try:
        names = open(obj + ".d").read().replace("\\\n", " ").split(":", 1)[1].split()
        age = os.path.getmtime(obj)
        return all(os.path.getmtime(n) <= age for n in names + [os.path.abspath(__file__)])
    except (OSError, IndexError):
        return False


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    newest = max(os.path.getmtime(p) for p in DEPS)
    key = _key(extra)
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= newest and not extra and not _other_flags(key):
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    inc = ["-I", os.path.join(ROOT, "include"), "-I", os.path.join(HERE, "csrc")]
    objs, running = [], []
    for src in SRCS:
        obj = os.path.join(OBJ_DIR, f"{os.path.basename(src)[:-3]}.{key}.o")
        objs.append(obj)
        if not force and not extra and _fresh(obj):
            continue
        tmp = obj + f".{os.getpid()}.tmp.o"  # a name of its own: two builds may run at once
        cmd = [NVCC, *FLAGS, *(extra or []), *inc, "-MD", "-MF", tmp + ".d", "-c", src, "-o", tmp]
        if verbose:
            print(" ".join(cmd), flush=True)
        running.append((cmd, tmp, obj, subprocess.Popen(cmd)))
    failed = None
    for cmd, tmp, obj, p in running:
        if p.wait() != 0:
            failed = failed or subprocess.CalledProcessError(p.returncode, cmd)
            continue
        os.replace(tmp + ".d", obj + ".d")
        os.replace(tmp, obj)
    if failed:
        raise failed
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [NVCC, *FLAGS, "-shared", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.check_call(cmd)
    with open(os.path.join(OBJ_DIR, "linked"), "w") as f:
        f.write(key)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None)
