"""Build ``libdecoderattn.so`` in-tree with nvcc for sm_103a (GB300).

Each translation unit compiles in parallel to an object under ``_build/``,
then one ``nvcc -shared`` links them (the CUDA runtime is linked statically,
so loading the library needs no CUDA shared object until a call reaches the
GPU).  No CMake, one ``-gencode``: a rebuild takes well under a minute.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import re
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libdecoderattn.so")
SOURCES = ["dr_api.cu", "attention.cu", "kv_append.cu", "sampler.cu", "heads.cu", "lm_head_tc.cu",
           "rope_append.cu", "attn_tokens.cu", "attn_tiles.cu", "dr_prompt_api.cu",
           "linear.cu", "linear_rows.cu", "linear_cluster.cu", "linear_tiles.cu", "residual_norm.cu", "dr_layer_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]

# Kernels that share a launch's registers out between their warps, and the registers per thread that they count on: a launch
# with another number is refused at run time, so the build looks at what ptxas gave them.
LAUNCH_REGISTERS = {"attn_tiles.cu": ("attn_tiles_kernel", 128), "linear_tiles.cu": ("linear_tiles_kernel", 96)}


def check_registers(src: str, ptxas: str) -> None:
    """Raise unless ptxas's report (-v) gives every kernel of LAUNCH_REGISTERS[src] its registers."""
    kernel, want = LAUNCH_REGISTERS[src]
    used = [(name, int(n)) for name, n in re.findall(r"entry function '(\w+)'.*?Used (\d+) registers", ptxas, flags=re.S)
            if kernel in name]
    bad = [f"{name}: {n}" for name, n in used if n != want]
    if bad or not used:
        raise RuntimeError(f"{src}: {kernel} needs {want} registers per thread, ptxas reports " + (", ".join(bad) or "none"))


def _nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(home, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _inputs_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return max(os.path.getmtime(f) for f in files)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile the library if it is missing or older than its sources; return its path."""
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _inputs_mtime():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        report = ["-Xptxas", "-v"] if src in LAUNCH_REGISTERS and "-v" not in flags else []
        cmd = [nvcc] + flags + report + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if src in LAUNCH_REGISTERS:
            check_registers(src, r.stdout + r.stderr)
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force=True, verbose=True, extra_flags=sys.argv[1:]))
