"""Builds libfa.so in-tree: every csrc/*.cu compiled for sm_103a in parallel, then linked; and
fa_torch.so, the torch binding of the small calls (csrc/fa_torch.cpp, host code), linked against it.

Usage: ``python -m tiled_attention_08_gb300.build [--verbose]``.  Object files and the
library go to ``tiled_attention_08_gb300/_build/`` (git-ignored).  A unit is recompiled when
it or any header it may include is newer than its object file.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libfa.so")
TORCH_SRC = os.path.join(CSRC, "fa_torch.cpp")
TORCH_LIB = os.path.join(BUILD, "fa_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _headers() -> list[str]:
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def _stale(obj: str, src: str, headers: list[str]) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(f) > t for f in [src, *headers])


def _compile(src: str, obj: str, verbose: bool) -> tuple[str, str]:
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return src, r.stdout + r.stderr


def _torch_dir() -> str | None:
    """Where torch is installed, or None."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    return list(spec.submodule_search_locations)[0]


def _compile_torch(obj: str) -> None:
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", inc, "-I",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-I", cuda, "-I",
           sysconfig.get_paths()["include"], "-c", TORCH_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for fa_torch.cpp:\n{r.stdout}\n{r.stderr}")


def _link_torch(obj: str) -> None:
    tmp = TORCH_LIB + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", os.path.join(_torch_dir(), "lib"), "-ltorch",
           "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_cuda", "-L", BUILD, "-l:libfa.so",
           "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of fa_torch.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TORCH_LIB)


def build(verbose: bool = False, force: bool = False) -> str:
    """Compiles and links the library and, where torch is installed, its binding; returns the path
    of libfa.so."""
    os.makedirs(BUILD, exist_ok=True)
    headers = _headers()
    torch_obj = os.path.join(BUILD, "fa_torch.o")
    torch_dir = _torch_dir()
    torch_job = None
    # Compiled by another torch than this one: its headers are part of the object's inputs.
    if torch_dir and (force or _stale(torch_obj, TORCH_SRC, [os.path.join(ROOT, "include", "fa.h"),
                                                             os.path.join(torch_dir, "version.py")])):
        torch_pool = cf.ThreadPoolExecutor(max_workers=1)
        torch_job = torch_pool.submit(_compile_torch, torch_obj)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    jobs = []
    for src in srcs:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        if force or verbose or _stale(obj, src, headers):
            jobs.append((src, obj))
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            for src, log in ex.map(lambda a: _compile(a[0], a[1], verbose), jobs):
                if verbose and log.strip():
                    print(f"== {os.path.basename(src)}\n{log}")
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    if jobs or not os.path.exists(LIB):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if not torch_dir:
        print("torch is not installed: fa_torch.so (decode_paged, rotary and the calls on a cache for torch "
              "tensors) is not built", file=sys.stderr)
        return LIB
    if torch_job is not None:
        torch_job.result()
    if torch_job is not None or not os.path.exists(TORCH_LIB):
        _link_torch(torch_obj)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force="--force" in sys.argv))
