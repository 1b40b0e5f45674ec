"""Build libpagedkv.so in-tree with nvcc for sm_103a.

Each .cu file compiles to an object in parallel; the objects link into
``paged_kv_cache_87_gb300/libpagedkv.so``.  ``_marshal.so`` beside it is the
binding's extension module (csrc/host/marshal.cc: torch tensors into calls of
the library), compiled by g++ at the same time.  The build is content-addressed: a
SHA-256 over every source and header, the compile and link flags and the
output of ``nvcc --version`` is stored beside the objects, and the library is
rebuilt whenever that digest changes (a modification time is never trusted).
"""
from __future__ import annotations

import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpagedkv.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedkv.so")
    return path


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _inputs() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        [os.path.join(ROOT, "include", "pagedkv.h"), __file__]


STAMP = os.path.join(BUILD, "libpagedkv.sha256")
LINK_FLAGS = ["-shared", "-cudart", "static"]
_nvcc_version: dict[str, str] = {}


def nvcc_version(cc: str) -> str:
    if cc not in _nvcc_version:
        r = subprocess.run([cc, "--version"], capture_output=True, text=True)
        _nvcc_version[cc] = r.stdout + r.stderr
    return _nvcc_version[cc]


def digest(extra_flags: list[str] | None = None, cc: str | None = None) -> str:
    """SHA-256 of what the library is built from: every input file (name and bytes),
    the architecture, compile and link flags, and the compiler's version string."""
    h = hashlib.sha256()
    for f in sorted(_inputs()):
        h.update(os.path.relpath(f, ROOT).encode() + b"\0")
        with open(f, "rb") as fh:
            h.update(fh.read())
        h.update(b"\0")
    for part in (ARCH, NVCC_FLAGS, extra_flags or [], LINK_FLAGS):
        h.update(("\x1f".join(part) + "\0").encode())
    h.update(nvcc_version(cc or nvcc()).encode())
    return h.hexdigest()


def up_to_date(extra_flags: list[str] | None = None) -> bool:
    if not os.path.exists(LIB) or not os.path.exists(STAMP):
        return False
    with open(STAMP) as f:
        return f.read().strip() == digest(extra_flags)


MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_SRC = os.path.join(CSRC, "host", "marshal.cc")
MARSHAL_STAMP = os.path.join(BUILD, "marshal.sha256")
GXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall"]


def _marshal_commands(obj: str, out: str) -> tuple[list[str], list[str]]:
    """The compile and link commands of the extension module, for the torch that runs this."""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    sysinc = [os.path.join(root, "include"),
              os.path.join(root, "include", "torch", "csrc", "api", "include"),
              os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")]
    abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    lib = os.path.join(root, "lib")
    built_for = f'-DPKV_TORCH="{torch.__version__}"'
    return (["g++", *GXX_FLAGS, abi, built_for, *[f"-I{i}" for i in inc],
             *[x for i in sysinc for x in ("-isystem", i)], "-c", MARSHAL_SRC, "-o", obj],
            ["g++", "-shared", "-o", out, obj, LIB, f"-L{lib}", "-ltorch_python", "-ltorch_cpu",
             "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"])


def _marshal_digest() -> str:
    import torch
    h = hashlib.sha256()
    for f in (MARSHAL_SRC, os.path.join(ROOT, "include", "pagedkv.h")):
        with open(f, "rb") as fh:
            h.update(fh.read() + b"\0")
    h.update(repr((_marshal_commands("o", "so"), torch.__version__, sys.version)).encode())
    return h.hexdigest()


def marshal_up_to_date() -> bool:
    if not os.path.exists(MARSHAL) or not os.path.exists(MARSHAL_STAMP):
        return False
    with open(MARSHAL_STAMP) as f:
        return f.read().strip() == _marshal_digest()


def _run(cmd: list[str], what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr}")
    return r.stderr


def build_marshal(compiled: str) -> None:
    """Link the compiled extension module against libpagedkv.so, in place."""
    tmp = MARSHAL + f".tmp{os.getpid()}"
    _run(_marshal_commands(compiled, tmp)[1], "linking _marshal.so")
    os.replace(tmp, MARSHAL)
    with open(MARSHAL_STAMP + f".tmp{os.getpid()}", "w") as f:
        f.write(_marshal_digest() + "\n")
    os.replace(MARSHAL_STAMP + f".tmp{os.getpid()}", MARSHAL_STAMP)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Build what is out of date of the library and the extension module."""
    os.makedirs(BUILD, exist_ok=True)
    obj = os.path.join(BUILD, "marshal.o")
    if not force and marshal_up_to_date():
        return build_library(force, verbose, ptxas_info)
    with ThreadPoolExecutor(max_workers=1) as ex:
        compiling = ex.submit(_run, _marshal_commands(obj, "")[0], "g++ on marshal.cc")
        lib = build_library(force, verbose, ptxas_info)
        compiling.result()
    build_marshal(obj)
    return lib


def build_library(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    if not force and up_to_date(extra):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    want = digest(extra, cc)

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(compile_one, sources()))
    if verbose or ptxas_info:
        for _, log in results:
            if log:
                print(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, *LINK_FLAGS, "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(STAMP + f".tmp{os.getpid()}", "w") as f:
        f.write(want + "\n")
    os.replace(STAMP + f".tmp{os.getpid()}", STAMP)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="-v" in sys.argv))
