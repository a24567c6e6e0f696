"""Build libmla_gb300.so in-tree with nvcc for sm_103a (no cmake).

Every translation unit under ``csrc/`` is compiled in parallel to an object
under ``_build/``; the objects are linked into
``mla_chunked_context_gb300/libmla_gb300.so`` (CUDA runtime linked statically,
so the library loads on a machine without a GPU).  ``csrc/py_decode.cpp``, the
decode calls' Python binding, becomes the module ``_decode`` beside it (its file
name says for which Python, its ``built_for`` for which PyTorch), with the host
compiler and the headers of Python and of the installed PyTorch.  The library
needs neither: ``build_library()`` makes it alone, and ``build()`` leaves it
built where the module fails.
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmla_gb300.so")
MODULE = os.path.join(HERE, "_decode" + sysconfig.get_config_var("EXT_SUFFIX"))
HEADER = os.path.join(HERE, "..", "include", "mla_chunked_context.h")
MODULE_SRC = os.path.join(CSRC, "py_decode.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", os.path.join(HERE, "..", "include")]


def nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found")
    return p


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith((".cu", ".cpp")) and f != os.path.basename(MODULE_SRC))


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip() and os.environ.get("MLA_BUILD_VERBOSE"):
        sys.stderr.write(r.stderr)
    return obj


def _run(what: str, cmd) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_module() -> str:
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    obj = os.path.join(BUILD, os.path.basename(MODULE_SRC) + ".o")
    _run(f"compiling {MODULE_SRC}", [
        "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
        f'-DMLA_BUILT_FOR="{torch.__version__}"',
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
        "-I", os.path.join(HERE, "..", "include"), "-isystem", inc,
        "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
        "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda,
        "-c", MODULE_SRC, "-o", obj])
    return obj


def _link_module(obj: str) -> None:
    import torch
    tmp = MODULE + ".tmp"
    _run("linking the Python module", [
        "g++", "-shared", "-o", tmp, obj, LIB, "-Wl,-rpath,$ORIGIN",
        "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu",
        "-lc10", "-lc10_cuda"])
    os.replace(tmp, MODULE)


def stale() -> bool:
    """The library or the module is missing, or older than a source."""
    srcs = [HEADER, *(os.path.join(CSRC, f) for f in os.listdir(CSRC))]
    newest = max(os.path.getmtime(p) for p in srcs)
    return any(not os.path.exists(p) or os.path.getmtime(p) < newest for p in (LIB, MODULE))


def build_library(extra_flags=()) -> str:
    """The C library alone."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, list(extra_flags)), srcs))
    tmp = LIB + ".tmp"
    _run("link", [nvcc(), *ARCH, "-shared", "-Xlinker", "-soname=" + os.path.basename(LIB), "-o", tmp,
                  *objs])
    os.replace(tmp, LIB)
    return LIB


def build(extra_flags=(), verbose: bool = False) -> str:
    """The library and the module, compiled side by side."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        module = ex.submit(_compile_module)
        build_library(extra_flags)
        _link_module(module.result())
    untagged = os.path.join(HERE, "_decode.so")  # of a build before the name said for which Python
    if os.path.exists(untagged):
        os.remove(untagged)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(sys.argv[1:], verbose=True)
