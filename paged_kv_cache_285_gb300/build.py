"""Build libpkv.so in-tree with nvcc for sm_103a.

Each .cu (and host-only .cpp) under csrc/ is compiled in parallel to an object under _build/, then
linked (static CUDA runtime) into paged_kv_cache_285_gb300/libpkv.so.  bind/calls.cpp, the binding
of the small calls, becomes _calls.so against libpkv.so and the installed torch; where that cannot
be built, a warning says so and the library stands without it.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libpkv.so")
CALLS_SRC = os.path.join(HERE, "bind", "calls.cpp")
CALLS = os.path.join(HERE, "_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-diag-suppress", "177",
         f"-I{INCLUDE}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpkv.so")


def _sources():
    # CUDA translation units and host-only C++ (compiled by nvcc's host compiler)
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _calls_cmd():
    """Object, compile command and torch's library folder for the binding; the object's name
    carries the torch it is compiled for."""
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    toolkit = os.path.dirname(os.path.dirname(nvcc()))
    obj = os.path.join(BUILD, f"calls-{torch.__version__}.o")
    return obj, [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", f"-I{INCLUDE}",
                 f"-I{root}/include", f"-I{root}/include/torch/csrc/api/include",
                 f"-I{toolkit}/include", f"-I{sysconfig.get_paths()['include']}",
                 f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                 f'-DPKV_TORCH_VERSION="{torch.__version__}"',
                 "-c", CALLS_SRC, "-o", obj], os.path.join(root, "lib")


def _link_calls(run, force, calls_obj, torch_lib, made):
    """Links _calls.so where it is not that object's; None, or what went wrong."""
    stamp = os.path.join(BUILD, "calls.linked")  # the object that _calls.so was linked from
    linked = ""
    if os.path.exists(stamp):
        with open(stamp) as f:
            linked = f.read()
    if not (force or made or linked != calls_obj or _stale(CALLS, [calls_obj, LIB])):
        return None
    tmp = CALLS + f".tmp{os.getpid()}"
    try:
        run([shutil.which("g++") or "g++", "-shared", calls_obj, "-o", tmp, f"-L{HERE}",
             "-l:libpkv.so", f"-L{torch_lib}", "-ltorch_python", "-ltorch_cpu", "-lc10",
             "-lc10_cuda", "-Wl,-rpath,$ORIGIN"])
    except (OSError, RuntimeError) as e:
        return e
    os.replace(tmp, CALLS)
    with open(stamp, "w") as f:
        f.write(calls_obj)
    return None


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    headers = _headers()
    jobs = []
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            jobs.append([cc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed on {cmd[-3]}")

    # The binding is optional (the package has the same calls through ctypes): what stands in its
    # way, a missing g++, Python.h or torch's headers, does not keep the library from being built.
    def compile_calls():
        try:
            calls_obj, calls_cmd, torch_lib = _calls_cmd()
            made = force or _stale(calls_obj, [CALLS_SRC] + glob.glob(os.path.join(INCLUDE, "*.h")))
            if made:
                run(calls_cmd)
            return calls_obj, torch_lib, made
        except (ImportError, OSError, RuntimeError) as e:
            return e

    with ThreadPoolExecutor(max_workers=min(len(jobs) + 1, os.cpu_count() or 4)) as ex:
        calls = ex.submit(compile_calls)
        list(ex.map(run, jobs))
        calls = calls.result()
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        run([cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    if not isinstance(calls, Exception):
        calls = _link_calls(run, force or bool(jobs), *calls)
    if isinstance(calls, Exception):
        for left in (CALLS, os.path.join(BUILD, "calls.linked")):  # made for another library
            if os.path.exists(left):
                os.remove(left)
        warnings.warn(f"_calls.so was not built ({calls}): the small calls go through ctypes")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
