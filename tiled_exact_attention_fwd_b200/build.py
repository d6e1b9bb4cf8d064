"""Build libfa.so (the C-ABI library) in-tree with nvcc for sm_100a.

Usage: python -m tiled_exact_attention_fwd_b200.build [--force] [--verbose]
Each .cu is compiled to an object in parallel, then linked into
tiled_exact_attention_fwd_b200/libfa.so (the CUDA runtime is linked statically). The Python
binding's marshalling for the operators around a paged cache (csrc/fa_torch.cpp, no device code)
is compiled with g++ against the installed torch into _fa_torch.so, which calls libfa.so.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfa.so")
BINDING = os.path.join(HERE, "_fa_torch.so")
BINDING_SOURCE = os.path.join(CSRC, "fa_torch.cpp")
SOURCES = ["fa_fwd.cu", "fa_fwd_paged.cu", "fa_bwd.cu", "fa_bwd256.cu", "fa_bwd_noalloc.cu", "fa_padding.cu",
           "fa_qk_norm.cu", "fa_chunk_rows.cu", "fa_chunk_tile.cu", "fa_key_weights.cu", "fa_key_weights_tile.cu",
           "fa_evict.cu", "fa_api.cu", "fa_cache_api.cu"]
HEADERS = ["fa_fwd_kernel.cuh", "fa_sync.cuh", "fa_seq.cuh", "fa_ptx.cuh", "fa_chunk.cuh", "fa_mma.cuh",
           "fa_internal.h"]

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newest_input() -> float:
    paths = [os.path.join(CSRC, s) for s in SOURCES + HEADERS] + [os.path.join(INCLUDE, "fa.h"),
                                                                   os.path.abspath(__file__)]
    return max(os.path.getmtime(p) for p in paths)


def _compile(src: str, verbose: bool, ptxas_v: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc()] + ARCH + FLAGS + (["-Xptxas", "-v"] if ptxas_v else []) + \
        ["-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if ptxas_v or verbose:
        sys.stdout.write(r.stderr)
    return obj


def _compile_binding(verbose: bool) -> str:
    import sysconfig

    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    obj = os.path.join(BUILD_DIR, "fa_torch.o")
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE]
    for d in (os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"], os.path.join(cuda, "include")):
        cmd += ["-isystem", d]
    cmd += ["-c", BINDING_SOURCE, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for fa_torch.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str, verbose: bool) -> None:
    import torch
    libs = os.path.join(os.path.dirname(os.path.abspath(torch.__file__)), "lib")
    tmp = BINDING + f".{os.getpid()}.tmp"
    # torch's libraries are loaded by the time this one is; libfa.so lies beside it
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:libfa.so", "-L", libs, "-lc10", "-ltorch", "-ltorch_cpu",
           "-ltorch_python", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def _binding_stale() -> bool:
    newest = max(os.path.getmtime(p) for p in (BINDING_SOURCE, os.path.join(INCLUDE, "fa.h"), os.path.abspath(__file__)))
    return not os.path.exists(BINDING) or os.path.getmtime(BINDING) < newest


def build(force: bool = False, verbose: bool = False, ptxas_v: bool = False) -> str:
    fresh = os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest_input()
    binding = force or _binding_stale()
    if not force and fresh and not binding:
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        pending = ex.submit(_compile_binding, verbose) if binding else None
        if force or not fresh:
            _link(list(ex.map(lambda s: _compile(s, verbose, ptxas_v), SOURCES)), verbose)
        if pending is not None:
            _link_binding(pending.result(), verbose)
    return LIB


def _link(objs: list, verbose: bool) -> None:
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [nvcc()] + ARCH + ["-shared", "-Xcompiler", "-fPIC", "-o", tmp] + objs + ["-lcuda"]
    # Link against the driver stub only for the CUtensorMap types' symbols if needed; the
    # tensor-map encoder itself is resolved at run time through the runtime's entry-point query.
    cmd = [c for c in cmd if c != "-lcuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv, ptxas_v="--ptxas-v" in sys.argv)
    print(LIB)
