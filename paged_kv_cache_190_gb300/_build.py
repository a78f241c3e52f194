"""Build of libpagedattn.so (in-tree, sm_103a only).

Each CUDA translation unit is compiled by nvcc in parallel with
``-gencode arch=compute_103a,code=sm_103a``; the host block manager by g++; the
objects are linked by nvcc into ``paged_kv_cache_190_gb300/libpagedattn.so``
(CUDA runtime linked statically, so the library loads on a machine without a
GPU driver and its block manager works there).  The per-step calls have a C++
binding for Python beside it, compiled by g++ against torch's headers and linked to
libpagedattn.so; its file name has the versions of torch and of the interpreter that it
serves.  A machine without torch or Python's headers builds the library alone.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpagedattn.so")
BINDING_SOURCE = os.path.join(CSRC, "step_binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CU_SOURCES = ["capi.cu", "cache_ops.cu", "decode_launch.cu", "decode_bf16.cu", "decode_f32.cu",
              "decode_fp8.cu", "decode_noalloc.cu", "cascade.cu", "rope_cache.cu", "capi_rope.cu",
              "span_launch.cu", "span_bf16.cu", "span_f32.cu", "span_fp8.cu", "span_fp4.cu",
              "capi_span.cu", "read_pages.cu", "prefill_launch.cu", "prefill_bf16.cu",
              "prefill_f32.cu", "capi_prefill.cu"]
CPP_SOURCES = ["block_manager.cpp", "cascade_groups.cpp"]


def _nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libpagedattn")
    return path


def _newer(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(os.path.dirname(PKG), "include", "pa.h"))
    return hs


def _no_binding():
    """Why the Python binding cannot be built here, or None."""
    try:
        import torch  # noqa: F401
    except (ImportError, OSError) as e:
        return f"torch cannot be imported ({e})"
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        return f"no Python.h in {include}"
    return None


def binding_path() -> str:
    """The Python binding for this interpreter and the torch that it imports."""
    import torch
    return os.path.join(PKG, f"_step.torch-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _binding_command(obj: str):
    """g++ over the binding's source, with the headers of the torch it will be used with."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    return ["g++", "-O2", "-std=c++17", "-fPIC", f"-I{root}/include",
            f"-I{root}/include/torch/csrc/api/include", f"-I{cuda}/include",
            f"-I{sysconfig.get_paths()['include']}",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-c", BINDING_SOURCE, "-o", obj]


def _binding_link(obj: str, out: str):
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++", "-shared", "-o", out, obj, f"-L{PKG}", "-l:libpagedattn.so", f"-L{lib}", "-lc10",
            "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link; returns the library path.  Skips up-to-date objects."""
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    headers = _headers()
    jobs = []
    objs = []
    for src in CU_SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OUT_DIR, src + ".o")
        objs.append(o)
        if force or _newer(o, [s] + headers):
            jobs.append([nvcc, *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
                         "-Xptxas", "-v" if verbose else "-O3", "-c", s, "-o", o])
    for src in CPP_SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OUT_DIR, src + ".o")
        objs.append(o)
        if force or _newer(o, [s] + headers):
            jobs.append(["g++", "-O2", "-std=c++17", "-fPIC", "-c", s, "-o", o])
    why_not = _no_binding()
    if why_not:
        print(f"libpagedattn: the Python binding of the per-step calls is not built: {why_not}", file=sys.stderr)
    else:
        binding = binding_path()
        binding_obj = os.path.join(OUT_DIR, os.path.basename(binding) + ".o")
        if force or _newer(binding_obj, [BINDING_SOURCE] + headers):
            jobs.insert(0, _binding_command(binding_obj))      # the longest of them first

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"build step failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return r.stderr if verbose else ""

    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        logs = list(ex.map(run, jobs))
    if verbose:
        for log in logs:
            if log:
                print(log)
    if jobs or force or not os.path.exists(LIB):
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    if not why_not and (force or _newer(binding, [binding_obj])):
        tmp = binding + f".tmp{os.getpid()}"
        run(_binding_link(binding_obj, tmp))
        os.replace(tmp, binding)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
