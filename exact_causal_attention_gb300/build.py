"""Builds the CUDA library in-tree with nvcc, sm_103a only."""
from __future__ import annotations

import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libeca_attn.so"
LIB_PATH = os.path.join(BUILD_DIR, LIB_NAME)
# The same sources with ECA_ANATOMY: the attention kernel records per-CTA milestone
# stamps (a measurement aid; nothing else changes).
ANATOMY_LIB_PATH = os.path.join(BUILD_DIR, "libeca_attn_anatomy.so")
SOURCES = ["attn_api.cu", "cache_api.cu", "prefill_api.cu", "mass_api.cu"]
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(home, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return files


def _flags(verbose: bool):
    return [*ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-cudart", "shared", "-I", INCLUDE,
            "-I", CSRC, *(["-Xptxas=-v"] if verbose else [])]


def _run(commands):
    """Run all commands at once; raise when one fails."""
    procs = [(subprocess.Popen(cmd), cmd) for cmd in commands]
    failed = [cmd for proc, cmd in procs if proc.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, " ".join(failed[0]))


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/ into _build/libeca_attn.so (and the anatomy variant beside it; all
    translation units in parallel) unless both are newer than every source.  Returns the
    main library."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    newest = max(os.path.getmtime(f) for f in _deps())
    libs = [(LIB_PATH, []), (ANATOMY_LIB_PATH, ["-DECA_ANATOMY"])]
    if not force and all(os.path.exists(path) and os.path.getmtime(path) >= newest for path, _ in libs):
        return LIB_PATH
    cuda_lib = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "lib64")
    tag = f".tmp{os.getpid()}"
    objects, compiles, links = [], [], []
    for path, defines in libs:
        mine = []
        for source in SOURCES:
            # Only the first source holds the attention kernel that the define changes.
            variant = os.path.basename(path) if source == SOURCES[0] else "shared"
            obj = os.path.join(BUILD_DIR, f"{source}.{variant}{tag}.o")
            if obj not in objects:
                objects.append(obj)
                compiles.append([_nvcc(), *_flags(verbose), *defines, "-c", os.path.join(CSRC, source), "-o", obj])
            mine.append(obj)
        links.append([_nvcc(), *ARCH_FLAGS, "--shared", "-cudart", "shared", "-Xlinker", f"-rpath,{cuda_lib}",
                      "-o", path + tag, *mine])
    try:
        _run(compiles)
        _run(links)
        for path, _ in libs:
            os.replace(path + tag, path)
    finally:
        for f in [*objects, *(path + tag for path, _ in libs)]:
            if os.path.exists(f):
                os.remove(f)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
