"""Build the in-tree CUDA library ``_build/libclef.so`` for sm_103a, and
``_build/clef_decode.so``, the compiled argument marshalling of ``decode.py``.

Each ``csrc/*.cu`` translation unit is compiled by nvcc in parallel
(``-gencode arch=compute_103a,code=sm_103a``) and the objects are linked
into one shared library against the shared CUDA runtime, so that it shares
the runtime instance (and the primary context) of the host process.  The
extension is one C++ file against the headers of Python and torch, linked to
libclef.so; it is built for one version of both and only where it is used, so
that a caller of the library alone needs nvcc and nothing else.
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
LIB = os.path.join(BUILD, "libclef.so")
EXT = os.path.join(BUILD, "clef_decode.so")
KEY = os.path.join(BUILD, "clef_decode.key")
ROOT = os.path.dirname(HERE)
SOURCES = ["abi.cu", "quant_act.cu", "gemm.cu", "swiglu.cu", "lora_noalloc.cu", "mma_peak.cu", "copy_sm.cu",
           "w4.cu", "kv_cache.cu", "kv_pages.cu", "kv_attention.cu"]
NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


EXT_SOURCE = "py_decode.cpp"
HEADER = os.path.join(ROOT, "include", "clef.h")


def _older(built, deps) -> bool:
    return not os.path.exists(built) or any(os.path.getmtime(d) > os.path.getmtime(built) for d in deps)


def _stale() -> bool:
    return _older(LIB, [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != EXT_SOURCE] + [HEADER])


def _ext_key() -> str:
    """What the extension is built against: this Python and this torch."""
    with open(os.path.join(_torch_dir(), "version.py"), encoding="utf-8") as f:
        return sys.version + "\n" + f.read()


def _ext_stale() -> bool:
    if _older(EXT, [os.path.join(CSRC, EXT_SOURCE), HEADER]) or not os.path.exists(KEY):
        return True
    with open(KEY, encoding="utf-8") as f:
        return f.read() != _ext_key()


def _run(what, cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _torch_dir() -> str:
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def _compile_extension() -> str:
    inc = os.path.join(_torch_dir(), "include")
    obj = os.path.join(BUILD, "py_decode.o")
    dirs = [os.path.join(ROOT, "include"), inc, os.path.join(inc, "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    _run(f"g++ on {EXT_SOURCE}", ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", *[a for d in dirs[:1] for a in ("-I", d)],
                                  *[a for d in dirs[1:] for a in ("-isystem", d)],
                                  "-c", os.path.join(CSRC, EXT_SOURCE), "-o", obj])
    return obj


def _link_extension(obj: str) -> None:
    """Against libclef.so beside it and the torch libraries that the process has loaded."""
    tmp = EXT + f".{os.getpid()}.tmp"
    _run("link of clef_decode.so", ["g++", "-shared", "-o", tmp, obj, "-L", BUILD, "-l:libclef.so", "-Wl,-rpath,$ORIGIN",
                                    "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
                                    "-lc10_cuda", "-lc10"])
    os.replace(tmp, EXT)
    tmp = KEY + f".{os.getpid()}.tmp"
    with open(tmp, "w", encoding="utf-8") as f:
        f.write(_ext_key())
    os.replace(tmp, KEY)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile library and extension (what is out of date of them) and return the path of libclef.so."""
    with ThreadPoolExecutor(max_workers=1) as ex:
        os.makedirs(BUILD, exist_ok=True)
        ext = ex.submit(_compile_extension) if force or _ext_stale() else None
        build_library(force, verbose)
        if ext:
            _link_extension(ext.result())
    return LIB


def build_extension() -> str:
    """The same for the extension alone, next to a built library."""
    if _ext_stale():
        os.makedirs(BUILD, exist_ok=True)
        _link_extension(_compile_extension())
    return EXT


def build_library(force: bool = False, verbose: bool = False) -> str:
    """The same for the library alone."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".{os.getpid()}.tmp"
    _run("link", [cc, "-shared", "-cudart", "shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
