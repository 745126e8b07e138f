"""Build libpagedattn.so in-tree with nvcc for sm_103a.

Each translation unit under ``csrc/`` is compiled in parallel, then linked into
``paged_kv_cache_55_gb300/libpagedattn.so``. Objects go to ``_build/`` next to
this file. ``csrc/native_binding.cpp`` becomes the Python extension ``_native``
beside it (g++, against the installed PyTorch's headers). Run
``python -m paged_kv_cache_55_gb300.build`` or call ``build()``.
"""

from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIBRARY = os.path.join(HERE, "libpagedattn.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
NATIVE = os.path.join(HERE, "_native" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libpagedattn.so")
    return path


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "pagedattn.h")]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    deps = _deps()
    if not force and not any(_stale(t, deps + [os.path.abspath(__file__)]) for t in (LIBRARY, NATIVE)):
        return LIBRARY
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    srcs = sources()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        native = ex.submit(compile_native)
        objs = list(ex.map(compile_one, srcs))
        native_obj = native.result()
    tmp = LIBRARY + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIBRARY)
    link_native(native_obj)
    return LIBRARY


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("PyTorch is not installed")
    return list(spec.submodule_search_locations)[0]


def _run(cmd, what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def compile_native() -> str:
    """Object file of the native marshalling module."""
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    obj = os.path.join(BUILD, "native_binding.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-isystem", inc, "-isystem",
          os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", sysconfig.get_paths()["include"],
          "-isystem", cuda, "-c", os.path.join(CSRC, "native_binding.cpp"), "-o", obj], "g++ on native_binding.cpp")
    return obj


def link_native(obj: str) -> None:
    """Linked to PyTorch's libraries and, by its path beside the module, to libpagedattn.so."""
    lib = os.path.join(_torch_dir(), "lib")
    tmp = NATIVE + ".tmp"
    _run(["g++", "-shared", obj, "-o", tmp, "-L", HERE, "-l:libpagedattn.so", "-Wl,-rpath,$ORIGIN", "-L", lib,
          f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"], "link of the native module")
    os.replace(tmp, NATIVE)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
