"""Build libvgemm.so (the C-ABI library) in-tree with nvcc for sm_103a.

Translation units are compiled in parallel, then linked into
``verify_gemm_gb300/_build/libvgemm.so``.  ``_vgtorch.so`` beside it, the calls
of the verify round from torch tensors, is compiled against the installed
torch by the host compiler and linked to it.  Run ``python -m
verify_gemm_gb300.build`` or call :func:`build`.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libvgemm.so")
TORCH_LIB = os.path.join(OUT_DIR, "_vgtorch.so")
TORCH_SOURCE = "vg_torch.cpp"
SOURCES = ["vg_api.cu", "vg_pack.cu", "vg_gemv.cu", "vg_noalloc.cu", "vg_probe.cu", "vg_rope.cu",
           "vg_attention.cu", "vg_attention_bf16.cu", "vg_attention_f16.cu", "vg_attention_e4m3.cu",
           "vg_attention_wide.cu", "vg_sample.cu"]
HEADERS = ["vg_device.cuh", "vg_internal.h", "vg_cache.h", "vg_attention.cuh", "vg_attention_wide.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-prec-div=true",
         "-prec-sqrt=true", "-ftz=false", "-fmad=true", f"-I{os.path.join(ROOT, 'include')}"]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libvgemm")
    return exe


def _stale() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(TORCH_LIB)):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(TORCH_LIB))
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS + [TORCH_SOURCE]]
    deps.append(os.path.join(ROOT, "include", "vgemm.h"))
    return any(os.path.getmtime(d) > t for d in deps)


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


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    exe = nvcc()
    objs = []

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

    with cf.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(compile_one, SOURCES))
        binding = binding.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [exe, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_binding(binding)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
