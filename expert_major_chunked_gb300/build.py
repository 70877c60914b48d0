"""Builds the CUDA library libmoe_prefill.so in-tree (expert_major_chunked_gb300/lib/) with nvcc for sm_103a.

Each .cu file is compiled on its own thread, then the objects are linked into one shared library (CUDA runtime
linked statically). attention_py.cpp, the Python extension through which `attention` calls that library with torch
tensors, is compiled beside them with g++ against torch's headers where torch is installed; the library itself needs
nothing of it. The extension is bound to the torch and the Python that it was compiled for, which a file beside it names.
"""

from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import threading
from concurrent.futures import ThreadPoolExecutor
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libmoe_prefill.so")
EXT_PATH = os.path.join(LIB_DIR, "attention_py.so")
EXT_KEY_PATH = os.path.join(LIB_DIR, "attention_py.key")
EXT_SOURCE = "attention_py.cpp"
SOURCES = ["gemm.cu", "gemm_pair.cu", "route.cu", "combine.cu", "combine_f64.cu", "ring.cu", "moe_prefill.cu", "noalloc.cu",
           "attention.cu", "attn_prefill.cu", "attn_decode.cu", "kv_cache.cu"]
HEADERS = ["internal.h", "ptx.cuh", "swiglu.cuh", "attn.h", "attn.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
_lock = threading.Lock()


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newer(output, inputs) -> bool:
    """Whether `output` is there and no input has changed since it was made."""
    if not os.path.exists(output):
        return False
    t = os.path.getmtime(output)
    return all(os.path.getmtime(f) <= t for f in [*inputs, os.path.abspath(__file__)])


def _headers():
    return [os.path.join(ROOT, "include", h) for h in ("moe_prefill.h", "moe_attention.h")]


def up_to_date() -> bool:
    return _newer(LIB_PATH, [os.path.join(CSRC, s) for s in SOURCES + HEADERS] + _headers())


def _torch_dir() -> Optional[str]:
    """Where torch is installed (located, not imported), or None."""
    try:
        spec = importlib.util.find_spec("torch")
    except ValueError:
        return None
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _extension_key() -> str:
    """What a compiled extension is bound to: Python's binary interface, torch's version and place."""
    torch_dir = _torch_dir()
    with open(os.path.join(torch_dir, "version.py")) as f:
        return f"{sysconfig.get_config_var('SOABI')}\n{torch_dir}\n{f.read()}"


def extension_up_to_date() -> bool:
    if not _newer(EXT_PATH, [os.path.join(CSRC, EXT_SOURCE)] + _headers()) or not os.path.exists(EXT_KEY_PATH):
        return False
    with open(EXT_KEY_PATH) as f:
        return f.read() == _extension_key()


def _run(cmd, what, show=False):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    if show:
        sys.stderr.write(r.stdout + r.stderr)


def _compile_extension(verbose: bool) -> str:
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    obj = os.path.join(LIB_DIR, "obj", "attention_py.o")
    includes = [sysconfig.get_paths()["include"], inc, os.path.join(inc, "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), os.path.join(ROOT, "include")]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-DNDEBUG", *[f"-I{p}" for p in includes], "-c",
          os.path.join(CSRC, EXT_SOURCE), "-o", obj], f"g++ on {EXT_SOURCE}", verbose)
    return obj


def _link_extension(obj: str) -> None:
    torch_lib = os.path.join(_torch_dir(), "lib")
    tmp = EXT_PATH + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, f"-L{torch_lib}", "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda",
          "-lc10", "-lc10_cuda", f"-L{LIB_DIR}", "-l:libmoe_prefill.so", "-Wl,-rpath,$ORIGIN"], "linking the extension")
    os.replace(tmp, EXT_PATH)
    with open(EXT_KEY_PATH, "w") as f:
        f.write(_extension_key())


def build_extension(force: bool = False, verbose: bool = False) -> str:
    """The extension alone, for a library that is there; returns its path."""
    with _lock:
        if _torch_dir() is None:
            raise RuntimeError("the attention operators work on torch tensors, and torch is not installed")
        if force or not extension_up_to_date():
            os.makedirs(os.path.join(LIB_DIR, "obj"), exist_ok=True)
            _link_extension(_compile_extension(verbose))
        return EXT_PATH


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False, extension: bool = True) -> str:
    """The library and, with `extension` and where torch is installed, the extension; returns the library's path."""
    with _lock:
        extension = extension and _torch_dir() is not None
        library = force or not up_to_date()
        extension = extension and (force or not extension_up_to_date())
        os.makedirs(os.path.join(LIB_DIR, "obj"), exist_ok=True)
        with ThreadPoolExecutor(max_workers=1) as ex:
            ext_obj = ex.submit(_compile_extension, verbose) if extension else None
            if library:
                _build_library(verbose, ptxas_info)
            if ext_obj:
                _link_extension(ext_obj.result())
        return LIB_PATH


def _build_library(verbose: bool, ptxas_info: bool) -> None:
    common = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "-I", os.path.join(ROOT, "include")]
    if ptxas_info:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(LIB_DIR, "obj", os.path.splitext(src)[0] + ".o")
        cmd = common + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
