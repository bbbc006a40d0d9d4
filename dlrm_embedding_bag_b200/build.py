"""Build the three libraries in-tree with nvcc for sm_100a.

``python -m dlrm_embedding_bag_b200.build`` (or ``__graft_entry__.build()``)
compiles every ``csrc/*.cu`` (the stage and its MLP layers), every
``csrc/tokens/*.cu`` (the token-level operators and the 8-bit layers) and every
``csrc/narrow/*.cu`` (the optimiser step and the 4-bit layers) to an object in
parallel and links ``libdlrm_sparse.so``, ``libdlrm_tokens.so`` and
``libdlrm_narrow.so`` next to this file. nvcc cross-compiles, so no GPU is needed.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
CSRC_TOKENS = os.path.join(CSRC, "tokens")
CSRC_NARROW = os.path.join(CSRC, "narrow")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libdlrm_sparse.so")
LIB_TOKENS = os.path.join(HERE, "libdlrm_tokens.so")
LIB_NARROW = os.path.join(HERE, "libdlrm_narrow.so")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler",
         "-fvisibility=hidden", "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.relpath(src, CSRC).replace(os.sep, "_") + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def _sources(d: str):
    return [p for p in glob.glob(os.path.join(d, "*")) if os.path.isfile(p)]


def _stale(lib: str, dirs) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = [p for d in dirs for p in _sources(d)] + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _link(lib: str, objs) -> None:
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile each CUDA library any of whose sources is newer; return the stage's path."""
    # the other libraries include headers of the stage's sources, the last one also the
    # token library's
    todo = [(lib, d) for lib, d, deps in ((LIB, CSRC, [CSRC]),
                                          (LIB_TOKENS, CSRC_TOKENS, [CSRC, CSRC_TOKENS]),
                                          (LIB_NARROW, CSRC_NARROW,
                                           [CSRC, CSRC_TOKENS, CSRC_NARROW]))
            if force or _stale(lib, deps)]
    if not todo:
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = [(lib, src) for lib, d in todo for src in sorted(glob.glob(os.path.join(d, "*.cu")))]
    with cf.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        objs = list(ex.map(lambda s: _compile(s[1], verbose), srcs))
    for lib, _ in todo:
        _link(lib, [o for (n, _), o in zip(srcs, objs) if n == lib])
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
