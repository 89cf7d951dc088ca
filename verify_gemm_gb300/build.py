"""Build libvgemm.so (the C-ABI library) in-tree with nvcc for sm_103a.

Translation units are compiled in parallel, then linked into
``verify_gemm_gb300/_build/libvgemm.so``.  ``_vgtorch.so`` beside it, the calls
of the verify round from torch tensors, is compiled against the installed
torch by the host compiler and linked to it.  Where that cannot be done (no
headers of torch's or Python's) the library is there all the same, with a
warning, and only the calls that need the binding raise.  Run ``python -m
verify_gemm_gb300.build`` or call :func:`build`.
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import fcntl
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libvgemm.so")
TORCH_LIB = os.path.join(OUT_DIR, "_vgtorch.so")
TORCH_SOURCE = "vg_torch.cpp"
SOURCES = ["vg_api.cu", "vg_pack.cu", "vg_gemv.cu", "vg_noalloc.cu", "vg_probe.cu", "vg_rope.cu",
           "vg_attention.cu", "vg_attention_bf16.cu", "vg_attention_f16.cu", "vg_attention_e4m3.cu",
           "vg_attention_wide.cu", "vg_sample.cu", "vg_norm_rope.cu", "vg_draw.cu",
           "vg_prefix.cu", "vg_attention_bf16_parts.cu", "vg_attention_f16_parts.cu", "vg_attention_e4m3_parts.cu",
           "vg_attention_wide_parts.cu"]
HEADERS = ["vg_device.cuh", "vg_internal.h", "vg_cache.h", "vg_pairs.cuh", "vg_rope.cuh", "vg_rows.cuh", "vg_attention.cuh",
           "vg_attention_wide.cuh", "vg_prefix.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-prec-div=true",
         "-prec-sqrt=true", "-ftz=false", "-fmad=true", f"-I{os.path.join(ROOT, 'include')}"]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libvgemm")
    return exe


def _older(target, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps + [os.path.join(ROOT, "include", "vgemm.h")])


def _stale() -> bool:
    return _older(LIB, [os.path.join(CSRC, f) for f in SOURCES + HEADERS])


def _made_for() -> str:
    """The torch and the Python whose headers the binding is compiled with."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"{_torch_dir()}\n{f.read()}\n{sysconfig.get_config_var('SOABI')}\n"


def _binding_stale() -> bool:
    # (kept beside the binding: an installed torch's files are older than it)
    try:
        with open(TORCH_LIB + ".for") as f:
            if f.read() != _made_for():
                return True
    except OSError:
        return True
    return _older(TORCH_LIB, [os.path.join(CSRC, TORCH_SOURCE)])


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _torch_dir() -> str:
    import importlib.util

    return os.path.dirname(importlib.util.find_spec("torch").origin)


def _cxx() -> str:
    exe = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if not exe:
        raise RuntimeError("no C++ compiler found for the torch binding")
    return exe


def _compile_binding() -> str:
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    obj = os.path.join(OUT_DIR, "vg_torch.o")
    _run([_cxx(), "-O2", "-std=c++20", "-fPIC", "-fvisibility=hidden", "-w", "-c",
          os.path.join(CSRC, TORCH_SOURCE), "-o", obj, f"-I{inc}",
          f"-I{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}",
          f"-I{sysconfig.get_paths()['include']}", f"-I{os.path.join(cuda, 'include')}"],
         "compiling the torch binding")
    return obj


def _link_binding(obj):
    lib = os.path.join(_torch_dir(), "lib")
    tmp = TORCH_LIB + f".tmp{os.getpid()}"
    _run([_cxx(), "-shared", "-o", tmp, obj, f"-L{OUT_DIR}", "-lvgemm", f"-L{lib}", "-lc10",
          "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN",
          f"-Wl,-rpath,{lib}"], "linking the torch binding")
    os.replace(tmp, TORCH_LIB)
    with open(TORCH_LIB + ".for", "w") as f:
        f.write(_made_for())


def _build_library(verbose):
    exe = nvcc()

    def compile_one(src):
        obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        cmd = [exe, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    _run([exe, *ARCH, "-shared", "-o", tmp, *objs], "link")
    os.replace(tmp, LIB)


@contextlib.contextmanager
def _alone():
    """One build at a time in the folder: a process that waited finds the work done."""
    os.makedirs(OUT_DIR, exist_ok=True)
    with open(os.path.join(OUT_DIR, ".lock"), "w") as f:
        fcntl.flock(f, fcntl.LOCK_EX)
        yield


# Why the binding could not be made: tried once a process.
_binding_failed = None


def _needed(force):
    return force or _stale(), _binding_failed is None and (force or _binding_stale())


def build(force: bool = False, verbose: bool = False) -> str:
    if any(_needed(force)):
        with _alone():
            _build(*_needed(force), verbose)
    return LIB


def _build(library, binding, verbose):
    global _binding_failed
    with cf.ThreadPoolExecutor(1) as ex:
        obj = ex.submit(_compile_binding) if binding else None
        if library:
            _build_library(verbose)
        if binding:
            try:
                _link_binding(obj.result())
            except Exception as e:
                _binding_failed = str(e)
                if os.path.exists(TORCH_LIB):             # one of other headers
                    os.remove(TORCH_LIB)
                warnings.warn("the calls of the verify round from torch tensors are not available: "
                              + _binding_failed, RuntimeWarning, stacklevel=3)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
