"""Build libkv4mla.so in place with nvcc for sm_103a (GB300), and the PyTorch
side of its *_gqa8 entry points, the extension module _kv4torch, with g++.

Each translation unit under ``csrc/`` is compiled in parallel with
``-gencode arch=compute_103a,code=sm_103a -O3 -lineinfo`` (IEEE division and
no fast-math, so the cache write stays bit-exact), then linked into a shared
library next to this file.  Run ``python -m bit_kv_cache_nvfp4_gb300.build``
or call :func:`build`.

The library needs nvcc alone (:func:`build_library`; where PyTorch is missing,
running this file builds just that): the extension is built beside it, stale by
itself, and one that does not build leaves the library in place.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libkv4mla.so")
TORCH_PATH = os.path.join(HERE, "_kv4torch.so")
TORCH_STAMP = os.path.join(BUILD_DIR, "torch_version")   # what _kv4torch.so was built with
TORCH_SOURCE = "kv4_torch.cpp"
SOURCES = ["kv4_capi.cu", "kv4_quantize_write.cu", "kv4_sparse_mla_decode.cu", "kv4_dcp.cu",
           "kv4_gqa8.cu", "kv4_gqa8_attention.cu"]
HEADERS = ["kv4_device.cuh", "kv4_gqa8_device.cuh", "kv4_launch.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkv4mla.so")


def _torch_version() -> str:
    import torch
    return torch.__version__


def _newest(sources) -> float:
    deps = [os.path.join(CSRC, f) for f in sources]
    deps.append(os.path.join(INCLUDE, "kv4mla.h"))
    deps.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in deps)


def _stale() -> bool:
    return not os.path.exists(LIB_PATH) or os.path.getmtime(LIB_PATH) < _newest(SOURCES + HEADERS)


def _torch_stale() -> bool:
    if not (os.path.exists(TORCH_PATH) and os.path.exists(TORCH_STAMP)):
        return True
    with open(TORCH_STAMP) as f:
        if f.read() != _torch_version():
            return True
    return os.path.getmtime(TORCH_PATH) < _newest([TORCH_SOURCE])


def _torch_object():
    """(object path, compile command, link flags) of the extension module."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    obj = os.path.join(BUILD_DIR, "kv4_torch.o")
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"], INCLUDE]
    compile_cmd = (["g++", "-O2", "-std=c++20", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
                   + [f for d in inc for f in ("-isystem" if d != INCLUDE else "-I", d)]
                   + ["-c", os.path.join(CSRC, TORCH_SOURCE), "-o", obj])
    link = ["-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
            "-L", HERE, "-l:libkv4mla.so", "-Wl,-rpath,$ORIGIN"]
    return obj, compile_cmd, link


def _start(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _finish(procs, verbose) -> None:
    """Wait for (source, process) pairs; raise if one failed."""
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if out and (verbose or p.returncode != 0):
            sys.stdout.write(out)
        if p.returncode != 0:
            failed.append(src)
    if failed:
        raise RuntimeError(f"compilation failed for {failed}")


def build_library(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile and link libkv4mla.so; returns its path."""
    if not force and not _stale():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++20", "-Xcompiler", "-fPIC,-O2",
                    "-I", INCLUDE, "-I", CSRC] + list(extra_flags or [])
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(obj)
        procs.append((src, _start([nvcc] + flags + ["-c", os.path.join(CSRC, src), "-o", obj], verbose)))
    _finish(procs, verbose)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def _link_extension(obj, link) -> None:
    tmp = TORCH_PATH + f".tmp{os.getpid()}"
    subprocess.run(["g++", "-shared", "-o", tmp, obj] + link, check=True)
    os.replace(tmp, TORCH_PATH)
    with open(TORCH_STAMP, "w") as f:
        f.write(_torch_version())


def build_extension(force: bool = False, verbose: bool = False) -> str:
    """Compile _kv4torch.so and link it to the library, which is there; returns
    its path."""
    if force or _torch_stale():
        os.makedirs(BUILD_DIR, exist_ok=True)
        obj, cmd, link = _torch_object()
        _finish([(TORCH_SOURCE, _start(cmd, verbose))], verbose)
        _link_extension(obj, link)
    return TORCH_PATH


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Both, their sources compiled side by side; returns the library's path."""
    ext = None
    if importlib.util.find_spec("torch") is not None and (force or _torch_stale()):
        os.makedirs(BUILD_DIR, exist_ok=True)
        obj, cmd, link = _torch_object()
        ext = [(TORCH_SOURCE, _start(cmd, verbose))]
    try:
        build_library(force, verbose, extra_flags)
    finally:
        if ext is not None:
            _finish(ext, verbose)
    if ext is not None:
        _link_extension(obj, link)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
