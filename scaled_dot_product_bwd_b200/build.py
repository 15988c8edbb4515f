"""Build the sm_100a shared libraries in-tree:

    scaled_dot_product_bwd_b200/libsdpa_b200.so         attention (csrc/)
    scaled_dot_product_bwd_b200/libsdpa_serve_b200.so   serving (csrc/serve/)
    scaled_dot_product_bwd_b200/_serve.so               its torch argument marshalling

    python -m scaled_dot_product_bwd_b200.build [--verbose]

nvcc cross-compiles for sm_100a without a GPU.  The CUDA runtime is linked
statically so the libraries need only the driver at run time.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libsdpa_b200.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
SOURCES = ["sdpa_api.cu"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps():
    out = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))]
    out.append(os.path.join(INCLUDE, "sdpa.h"))
    return out


def _source_hash(flags) -> str:
    import hashlib
    h = hashlib.sha256(" ".join(flags).encode())
    for d in sorted(_deps()):
        if os.path.isfile(d):
            h.update(os.path.relpath(d, ROOT).encode())
            with open(d, "rb") as fh:
                h.update(fh.read())
    return h.hexdigest()


FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-gencode", "arch=compute_100a,code=sm_100a",
         "-Xcompiler", "-fPIC", "-shared", "-cudart", "static"]


def source_hash() -> str:
    """Hash of the kernel sources and build flags the library is built from."""
    return _source_hash(FLAGS)


SERVE_CSRC = os.path.join(CSRC, "serve")
SERVE_LIB_PATH = os.path.join(PKG, "libsdpa_serve_b200.so")
SERVE_BIND_PATH = os.path.join(PKG, "_serve.so")


def _serve_deps():
    return sorted(_deps() + [os.path.join(SERVE_CSRC, f) for f in os.listdir(SERVE_CSRC)]
                  + [os.path.join(INCLUDE, "sdpa_serve.h")])


def _bind_flags():
    """g++ flags of the torch marshalling module."""
    import sysconfig

    import torch
    root = os.path.join(os.path.dirname(torch.__file__))
    inc = [os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_path("include"), os.path.join(os.path.dirname(os.path.dirname(nvcc_path())),
                                                       "include"), INCLUDE]
    return (["-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
            + [x for i in inc for x in ("-isystem" if "sdpa" not in i and i != INCLUDE else "-I", i)],
            ["-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch", "-ltorch_cpu", "-lc10",
             "-lc10_cuda", "-L" + PKG, "-l:libsdpa_serve_b200.so", "-Wl,-rpath,$ORIGIN"])


def _hash(paths, flags) -> str:
    import hashlib
    h = hashlib.sha256(" ".join(flags).encode())
    for d in paths:
        if os.path.isfile(d):
            h.update(os.path.relpath(d, ROOT).encode())
            with open(d, "rb") as fh:
                h.update(fh.read())
    return h.hexdigest()


def _make(out: str, stamp: str, cmd, verbose: bool, force: bool):
    """Run cmd -o out unless out was built with this stamp."""
    path = out + ".stamp"
    if not force and os.path.exists(out) and os.path.exists(path):
        with open(path) as fh:
            if fh.read().strip() == stamp:
                return
    r = subprocess.run(cmd + ["-o", out + ".tmp"], capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"building {os.path.basename(out)} failed")
    if verbose:
        sys.stderr.write(r.stderr)
    os.replace(out + ".tmp", out)
    with open(path, "w") as fh:
        fh.write(stamp + "\n")


def _build_serve(verbose: bool, force: bool):
    nvcc = [nvcc_path()] + FLAGS + (["-Xptxas=-v"] if verbose else [])
    _make(SERVE_LIB_PATH, _hash(_serve_deps(), FLAGS),
          nvcc + ["-I", INCLUDE, "-I", CSRC, os.path.join(SERVE_CSRC, "serve_api.cu")], verbose, force)
    flags, libs = _bind_flags()
    src = os.path.join(SERVE_CSRC, "serve_bind.cpp")
    _make(SERVE_BIND_PATH, _bind_stamp(flags + libs),
          [shutil.which("g++") or "g++"] + flags + [src] + libs, verbose, force)


def _bind_stamp(flags) -> str:
    """Of the marshalling module: its sources and flags, and the torch and Python whose
    headers and ABI it is compiled against (an upgrade in place changes no path)."""
    import torch
    deps = [os.path.join(SERVE_CSRC, "serve_bind.cpp"), os.path.join(INCLUDE, "sdpa.h"),
            os.path.join(INCLUDE, "sdpa_serve.h")]
    return _hash(deps, flags + [torch.__version__, str(torch.version.git_version), sys.version])


def build(verbose: bool = False, force: bool = False) -> str:
    from concurrent.futures import ThreadPoolExecutor
    with ThreadPoolExecutor(2) as pool:
        jobs = [pool.submit(_build_attention, verbose, force),
                pool.submit(_build_serve, verbose, force)]
        for j in jobs:
            j.result()
    return LIB_PATH


def _build_attention(verbose: bool, force: bool):
    cmd = [nvcc_path()] + FLAGS + (["-Xptxas=-v"] if verbose else []) + [
        "-I", INCLUDE, "-I", CSRC] + [os.path.join(CSRC, s) for s in SOURCES]
    _make(LIB_PATH, _source_hash(FLAGS), cmd, verbose, force)


if __name__ == "__main__":
    build(verbose="--verbose" in sys.argv, force=True)
    print(LIB_PATH, SERVE_LIB_PATH, SERVE_BIND_PATH)
