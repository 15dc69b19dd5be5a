"""Build libpa.so (the CUDA library behind include/pa.h) for sm_103a.

Each translation unit under csrc/ is compiled by its own nvcc process, in
parallel, then linked into one shared library with the CUDA runtime linked
statically.  Beside it the C++ part of the Python binding (pa_bind.cpp) is
compiled with g++ against the installed torch's headers.  Outputs (git-ignored):
<package>/_build/libpa.so and <package>/_build/pa_bind-<torch's version><Python's suffix
of extension modules>, .cpython-312-x86_64-linux-gnu.so for instance.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libpa.so")
# (of one torch, whose tensors it looks into, and of one Python: it is loaded by this path,
# which the import system's own check of the suffix does not see)
BIND = os.path.join(OUT_DIR, f"pa_bind-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")
SOURCES = ("pa_api.cu", "pa_blocks.cu", "pa_cache.cu", "pa_cache_fp4.cu", "pa_decode.cu",
           "pa_decode_fp4.cu", "pa_decode_sparse.cu", "pa_prefill_fp4.cu", "pa_prefill_tc.cu",
           "pa_rope.cu", "pa_sparse.cu", "pa_static_ws.cu")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libpa")
    return path


def _stale(out: str, *endings: str) -> bool:
    """Whether `out` is missing, or older than pa.h or a file of csrc/ with one of the endings."""
    if not os.path.exists(out):
        return True
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(endings)]
    deps.append(os.path.join(os.path.dirname(HERE), "include", "pa.h"))
    return any(os.path.getmtime(d) > os.path.getmtime(out) for d in deps)


def _run(what: str, cmd) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _torch_dir() -> str:
    return os.path.dirname(torch.__file__)


def _compile_bind(src: str, obj: str) -> None:
    inc = os.path.join(_torch_dir(), "include")
    _run("g++ on pa_bind.cpp", [
        "g++", "-std=c++17", "-O2", "-fPIC", "-Wall",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-isystem", inc,
        "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
        "-isystem", sysconfig.get_paths()["include"], "-I", CSRC, "-c", src, "-o", obj])


def _link_bind(obj: str, lib_dir: str, out: str) -> None:
    """`out` from `obj` and the libpa.so of lib_dir, which it looks for beside itself."""
    _run("link of the binding", ["g++", "-shared", "-o", out, obj, "-L" + lib_dir, "-l:libpa.so",
                                "-L" + os.path.join(_torch_dir(), "lib"), "-lc10", "-ltorch_cpu",
                                "-ltorch_python", "-Wl,-rpath,$ORIGIN"])


def _build_lib(verbose: bool) -> None:
    cc = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
        cmd = [cc, *FLAGS, *ARCH, "-c", os.path.join(CSRC, src), "-o", obj]
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
    _run("link", [cc, "-shared", *ARCH, "-o", tmp, *objs, "-cudart", "static"])
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    """Makes what is missing or older than its sources: the library, and the binding,
    which links against it but holds nothing of it."""
    lib = force or _stale(LIB, ".cu", ".cuh", ".h")
    bind = force or _stale(BIND, ".cpp")
    os.makedirs(OUT_DIR, exist_ok=True)
    bind_obj = os.path.join(OUT_DIR, "pa_bind.o")
    with ThreadPoolExecutor(max_workers=1) as ex:
        if bind:
            compiled = ex.submit(_compile_bind, os.path.join(CSRC, "pa_bind.cpp"), bind_obj)
        if lib:
            _build_lib(verbose)
        if bind:
            tmp = BIND + f".{os.getpid()}.tmp"
            try:  # (what follows needs the headers of Python and torch, which libpa.so does not)
                compiled.result()
                _link_bind(bind_obj, OUT_DIR, tmp)
            except (OSError, RuntimeError) as e:
                raise RuntimeError(f"{LIB} is built; the Python binding of rotated append and sparse "
                                   f"attention is not: {e}") from e
            os.replace(tmp, BIND)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
