"""Builds ``libpagedattn.so`` from ``csrc/`` with nvcc for sm_103a.

Each translation unit is compiled in parallel, then linked into one shared
library under ``paged_kv_cache_239_gb300/_build/``.  Only one ``-gencode``
(sm_103a) is emitted.  Beside it, for the installed Python and torch, the module
``pagedcalls`` (``pa_calls.cpp``), which calls the library, and a stamp that names both.
"""
from __future__ import annotations

import contextlib
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from typing import Optional

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(REPO_DIR, "include")
OUT_DIR = os.path.join(PKG_DIR, "_build")
LIB_NAME = "libpagedattn.so"
LIB_PATH = os.path.join(OUT_DIR, LIB_NAME)

CALLS_NAME = "pagedcalls.so"
CALLS_PATH = os.path.join(OUT_DIR, CALLS_NAME)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = ["pa_api.cpp", "pa_aux.cu", "pa_decode_bf16.cu", "pa_decode_f32.cu",
           "pa_decode_noalloc.cu", "pa_alloc.cu", "pa_decode_mma.cu",
           "pa_decode_mma_wide.cu", "pa_decode_umma.cu", "pa_rope.cu",
           "pa_prefill_mma.cu", "pa_prefill_umma.cu", "pa_pages.cu", "pa_plan.cu",
           "pa_tree_mma.cu", "pa_tree_mma_bf16.cu", "pa_tree_mma_f32.cu", "pa_tree_umma.cu",
           "pa_tree_umma_f32.cu",
           "pa_accept.cu"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedattn")
    return cand


def _older(path: str, files) -> bool:
    """Whether ``path`` is missing or older than one of the files."""
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(f) > t for f in files)


def _library_stale() -> bool:
    return _older(LIB_PATH, [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "pa_calls.cpp"]
                  + [os.path.join(INCLUDE, "pagedattn.h")])


def _torch_dir() -> Optional[str]:
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def calls_need() -> str:
    """What the module cannot be built without and is not there ("": nothing).  The library, which
    C programs use by itself, needs none of it."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        return "torch"
    if not (os.path.exists(os.path.join(torch_dir, "include", "c10", "cuda", "CUDAStream.h"))
            and os.path.exists(os.path.join(torch_dir, "lib", "libc10_cuda.so"))):
        return "a torch for CUDA, with its headers"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers"
    return ""


def _installed_torch() -> str:
    """The version of the torch on the disk (found without importing torch, which takes
    longer than the rest of the build on a cold machine)."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return re.search(r"^__version__ = ['\"](.*?)['\"]", f.read(), re.M).group(1)


def _python_abi() -> str:
    return sysconfig.get_config_var("SOABI")


def calls_stamp(torch_version: str) -> str:
    """What the module is bound to, as the file beside it says."""
    return f"torch {torch_version}, {_python_abi()}"


def read_calls_stamp() -> str:
    try:
        with open(CALLS_PATH + ".stamp") as f:
            return f.read()
    except OSError:
        return "no known torch"


def _calls_stale() -> bool:
    """Older than its source, or for another torch (on the disk, or in this process) or Python;
    False where it cannot be built."""
    if calls_need():
        return False
    if _older(CALLS_PATH, [os.path.join(CSRC, "pa_calls.cpp"), os.path.join(INCLUDE, "pagedattn.h")]):
        return True
    stamp = read_calls_stamp()
    loaded = sys.modules.get("torch")
    return stamp != calls_stamp(_installed_torch()) or (
        loaded is not None and stamp != calls_stamp(str(loaded.__version__)))


def _stale() -> bool:
    return _library_stale() or _calls_stale()


def _compile_calls() -> str:
    """The object of the Python module."""
    inc = os.path.join(_torch_dir(), "include")
    obj = os.path.join(OUT_DIR, "pa_calls.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include"),
           "-c", os.path.join(CSRC, "pa_calls.cpp"), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for pa_calls.cpp:\n{res.stdout}\n{res.stderr}")
    return obj


def _link_calls(obj: str) -> None:
    torch_lib = os.path.join(_torch_dir(), "lib")
    stamp = calls_stamp(_installed_torch())
    tmp = CALLS_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", OUT_DIR, "-lpagedattn", "-Wl,-rpath,$ORIGIN",
           "-L", torch_lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           f"-Wl,-rpath,{torch_lib}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    if read_calls_stamp() == stamp:
        os.replace(tmp, CALLS_PATH)
        return
    # no module stands beside another one's stamp
    with contextlib.suppress(FileNotFoundError):
        os.remove(CALLS_PATH + ".stamp")
    os.replace(tmp, CALLS_PATH)
    with open(tmp, "w") as f:
        f.write(stamp)
    os.replace(tmp, CALLS_PATH + ".stamp")


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link what is missing or stale of the library and, where it can be built
    (``calls_need``), the module; returns the library's path.  Raises on failure."""
    library, module = force or _library_stale(), _calls_stale() or (force and not calls_need())
    if not library and not module:
        return LIB_PATH
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    common = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "-I", INCLUDE, "-I", CSRC,
              *ARCH, *extra_flags]
    if verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src: str) -> str:
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
        lang = ["-x", "cu"] if src.endswith(".cu") else []
        cmd = [nvcc, *common, *lang, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
        if verbose and (res.stdout or res.stderr):
            print(res.stdout + res.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(_compile_calls) if module else None
        objs = list(ex.map(compile_one, SOURCES)) if library else []
    if library:
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-lrt", "-ldl", "-lpthread"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB_PATH)
    if calls is not None:
        _link_calls(calls.result())
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
    if calls_need():
        print(f"{CALLS_NAME} was not built: it needs {calls_need()}")
