"""Build libduo_kv.so in-tree for sm_100a with nvcc, and the compiled half of
the Python binding (_binding.so) with g++ against torch's headers.  Without
torch only the library is built: a C program needs no more.

    python -m head_wise_kv_b200.build          # incremental
    python -m head_wise_kv_b200.build --force  # rebuild everything
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(ROOT, "_build", "duo_kv")
LIB = os.path.join(PKG, "libduo_kv.so")
BINDING_SRC = os.path.join(CSRC, "bindings.cpp")
BINDING = os.path.join(PKG, "_binding.so")
BUILT_FOR = os.path.join(OBJDIR, "_binding.built_for")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    cc = nvcc()
    hdr_mtime = max(os.path.getmtime(h) for h in _headers())
    objs, rebuilt = [], False
    for src in _sources():
        obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if (not force and os.path.exists(obj) and os.path.getmtime(obj) >= os.path.getmtime(src)
                and os.path.getmtime(obj) >= hdr_mtime):
            continue
        cmd = [cc, *ARCH, *FLAGS, *(extra or []), "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        rebuilt = True
    if force or rebuilt or not os.path.exists(LIB) or any(
            os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        cmd = [cc, *ARCH, "-shared", "-o", LIB, *objs, "-cudart", "static"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    if importlib.util.find_spec("torch") is not None:
        build_binding(force, verbose)
    else:
        print("head_wise_kv_b200: no torch, so no Python binding: built the C library alone", file=sys.stderr)
    return LIB


def built_for() -> str:
    """What _binding.so depends on besides its sources: the Python and torch that it was built against."""
    import importlib.metadata
    spec = importlib.util.find_spec("torch")
    return f"python {sys.version}\ntorch {importlib.metadata.version('torch')} {spec.origin}\n"


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """_binding.so: links libduo_kv.so beside it and the torch that is installed."""
    inputs = [BINDING_SRC, os.path.join(INCLUDE, "duo_kv.h")]
    stamp = built_for()
    if not force and os.path.exists(BINDING) and all(os.path.getmtime(BINDING) >= os.path.getmtime(f) for f in inputs):
        if os.path.exists(BUILT_FOR):
            with open(BUILT_FOR) as f:
                if f.read() == stamp:
                    return BINDING
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    home = os.path.dirname(os.path.dirname(nvcc()))
    libs = cpp_extension.library_paths()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-DTORCH_EXTENSION_NAME=_binding",
           "-DTORCH_API_INCLUDE_EXTENSION_H", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-I{INCLUDE}", *[f"-isystem{d}" for d in cpp_extension.include_paths()],
           f"-isystem{sysconfig.get_path('include')}", f"-isystem{home}/include", BINDING_SRC, "-o", BINDING,
           *[f"-L{d}" for d in libs], "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python",
           f"-L{PKG}", "-l:libduo_kv.so", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.makedirs(OBJDIR, exist_ok=True)
    with open(BUILT_FOR, "w") as f:
        f.write(stamp)
    return BINDING


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print register / shared-memory use")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_info else None
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose, extra=extra))


if __name__ == "__main__":
    sys.exit(main())
