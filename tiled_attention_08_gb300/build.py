"""Builds libfa.so in-tree: every csrc/*.cu compiled for sm_103a in parallel, then linked; and
fa_torch.so, the torch binding of the small calls (csrc/fa_torch.cpp, host code), linked against it.

Usage: ``python -m tiled_attention_08_gb300.build [--verbose]``.  Object files and the
library go to ``tiled_attention_08_gb300/_build/`` (git-ignored).  A unit is recompiled when
it or any header it may include is newer than its object file (the binding also when the
installed torch is not the one it was compiled for), and a library is linked again when an
object is newer than it.  Objects and libraries are put in place whole, so that an interrupted
build leaves none that looks fresh.
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


def _run(cmd: list[str], out: str, what: str) -> str:
    """Runs a command that writes ``out``, which appears whole or not at all; returns its messages."""
    tmp = out + f".tmp{os.getpid()}"
    r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        if os.path.exists(tmp):
            os.remove(tmp)
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    return r.stdout + r.stderr


def _compile(src: str, obj: str, verbose: bool) -> tuple[str, str]:
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, "-c", src]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    return src, _run(cmd, obj, f"nvcc failed for {os.path.basename(src)}")


def _torch_dir() -> str | None:
    """Where torch is installed, or None."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    return list(spec.submodule_search_locations)[0]


def _torch_id() -> str:
    """The installed torch that an object was compiled for: its place and its version file."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return _torch_dir() + "\n" + f.read()


def _other_torch(note: str) -> bool:
    """Whether the note beside the object names another torch than the installed one."""
    if not os.path.exists(note):
        return True
    with open(note) as f:
        return f.read() != _torch_id()


def _compile_torch(obj: str, note: str) -> None:
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    if os.path.exists(note):  # (no note: compiled again, should this end half way)
        os.remove(note)
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", inc, "-I",
          os.path.join(inc, "torch", "csrc", "api", "include"), "-I", cuda, "-I",
          sysconfig.get_paths()["include"], "-c", TORCH_SRC], obj, "g++ failed for fa_torch.cpp")
    with open(note, "w") as f:
        f.write(_torch_id())


def _link_torch(obj: str) -> None:
    _run(["g++", "-shared", obj, "-L", os.path.join(_torch_dir(), "lib"), "-ltorch", "-ltorch_cpu",
          "-ltorch_python", "-lc10", "-lc10_cuda", "-L", BUILD, "-l:libfa.so", "-Wl,-rpath,$ORIGIN"],
         TORCH_LIB, "link of fa_torch.so failed")


def build(verbose: bool = False, force: bool = False) -> str:
    """Compiles and links the library and, where torch is installed, its binding; returns the path
    of libfa.so."""
    os.makedirs(BUILD, exist_ok=True)
    headers = _headers()
    torch_obj = os.path.join(BUILD, "fa_torch.o")
    torch_note = torch_obj + ".torch"
    torch_dir = _torch_dir()
    torch_job = None
    if torch_dir and (force or _other_torch(torch_note) or
                      _stale(torch_obj, TORCH_SRC, [os.path.join(ROOT, "include", "fa.h")])):
        torch_pool = cf.ThreadPoolExecutor(max_workers=1)
        torch_job = torch_pool.submit(_compile_torch, torch_obj, torch_note)
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
    if _stale(LIB, objs[0], objs):
        _run([_nvcc(), *ARCH, "-shared", *objs], LIB, "link failed")
    if not torch_dir:
        print("torch is not installed: fa_torch.so (decode_paged, rotary and the calls on a cache for torch "
              "tensors) is not built", file=sys.stderr)
        return LIB
    if torch_job is not None:
        torch_job.result()
    if _stale(TORCH_LIB, torch_obj, []):
        _link_torch(torch_obj)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force="--force" in sys.argv))
