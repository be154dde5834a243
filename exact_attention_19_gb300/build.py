"""Build libfa_gb300.so in-tree with nvcc (sm_103a only).

Six translation units: fa_api.cu (the C-ABI front end with every dense
forward, split-KV merge and backward kernel instantiation), fa_rope.cu (rotary
positions, with the norm of each head or without, and the paged cache's append),
fa_paged.cu (attention over the paged cache), fa_cache.cu (the weight that cached
keys gather, and eviction), fa_probe.cu (the exp2-throughput probe) and fa_selftest.cu (the
bounded-wait self-test), compiled in parallel by one nvcc call; beside them
fa_torch, the host-side fast path of the torch entry points (fa_torch.cpp, the
host compiler against torch's headers; its file is named after the torch and
Python it was compiled for).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libfa_gb300.so")
SOURCES = [os.path.join(CSRC, f) for f in ("fa_api.cu", "fa_rope.cu", "fa_paged.cu", "fa_cache.cu", "fa_probe.cu",
                                              "fa_selftest.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in ("fa_ptx.cuh", "fa_host.h", "fa_fwd_kernel.cuh", "fa_fwd_persist.cuh",
                                                       "fa_bwd_kernel.cuh", "fa_rope_kernel.cuh", "fa_norm_kernel.cuh",
                                                       "fa_paged_kernel.cuh", "fa_paged_tile.cuh",
                                                       "fa_cache_ptx.cuh",
                                                       "fa_weights_kernel.cuh", "fa_evict_kernel.cuh")] + [
    os.path.join(INCLUDE, "fa.h")]

TORCH_SOURCE = os.path.join(CSRC, "fa_torch.cpp")
TORCH_DEPS = [TORCH_SOURCE, os.path.join(INCLUDE, "fa.h")]

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfa_gb300.so")
    return path


def command(out: str = LIB_PATH, verbose_ptxas: bool = False) -> list[str]:
    cmd = [nvcc(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "--threads=0", "-shared", "-Xcompiler", "-fPIC",
           "-I", INCLUDE, "-I", CSRC, "-o", out, *SOURCES, "-lcudart"]
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    return cmd


def torch_lib_path() -> str:
    """Where the torch module for the running interpreter and torch lies.  It is compiled against torch's
    C++ classes, so each version of either has a file of its own and never loads another's."""
    import sysconfig

    import torch

    return os.path.join(LIB_DIR, f"fa_torch.{torch.__version__}.cxx11abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
                                 f"{sysconfig.get_config_var('EXT_SUFFIX') or '.so'}")


def torch_command(out: str) -> list[str]:
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"],
           os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")]
    lib = os.path.join(root, "lib")
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
            *[x for d in inc for x in ("-isystem", d)], "-o", out, TORCH_SOURCE, "-L", lib, f"-Wl,-rpath,{lib}",
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _stale(out: str, deps: list[str]) -> bool:
    return not os.path.exists(out) or any(os.path.getmtime(f) > os.path.getmtime(out) for f in deps)


def needs_build() -> bool:
    if _stale(LIB_PATH, DEPS):
        return True
    try:
        return _stale(torch_lib_path(), TORCH_DEPS)
    except Exception:  # without torch there is no module to build
        return False


def _start(out: str, cmd: list[str]):
    return out, cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)


def _finish(job, tmp: str, echo: bool) -> str:
    """Wait for a compiler and put its output in place; what went wrong, or an empty text."""
    out, cmd, proc = job
    stdout, stderr = proc.communicate()
    if proc.returncode != 0:
        return f"{cmd[0]} failed:\n{stdout}\n{stderr}"
    if echo:
        sys.stderr.write(stderr)
    os.replace(tmp, out)
    return ""


def build(force: bool = False, verbose_ptxas: bool = False, strict: bool = False) -> str:
    """Compile what is out of date (both libraries at once); the path of libfa_gb300.so.

    The C ABI needs no torch: where torch is missing, or fa_torch does not compile against it,
    libfa_gb300.so is built all the same, with a note on stderr (the torch entry points raise at their
    first use); ``strict`` raises instead, once libfa_gb300.so is in place.
    """
    os.makedirs(LIB_DIR, exist_ok=True)
    suffix = f".tmp{os.getpid()}"
    lib_job = torch_job = None
    if force or _stale(LIB_PATH, DEPS):
        lib_job = _start(LIB_PATH, command(LIB_PATH + suffix, verbose_ptxas))
    torch_failure = ""
    try:
        torch_path = torch_lib_path()
        if force or _stale(torch_path, TORCH_DEPS):
            torch_job = _start(torch_path, torch_command(torch_path + suffix))
    except Exception as e:  # no torch, a torch that does not load, no host compiler
        torch_failure = f"{type(e).__name__}: {e}"
    failure = _finish(lib_job, LIB_PATH + suffix, verbose_ptxas) if lib_job else ""
    if torch_job:
        torch_failure = _finish(torch_job, torch_path + suffix, verbose_ptxas)
    if failure:
        raise RuntimeError("\n".join(x for x in (failure, torch_failure) if x))
    if torch_failure:
        if strict:
            raise RuntimeError(f"fa_torch was not built: {torch_failure}")
        sys.stderr.write(f"fa_torch (the torch entry points rope, norm_rope, kv_append, fwd_paged, "
                         f"fwd_prefix, kv_weights, kv_evict) was not built: "
                         f"{torch_failure}\n")
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv)
    print(LIB_PATH)
