"""Build libtq.so (the C-ABI library) in-tree with nvcc for sm_100a, and _bind.so (the compiled part of its Python
binding) against the installed torch.

Usage: ``python -m kv_cache_vector_norm_b200._build [--force] [--verbose]``.  The library is rebuilt when any of its
sources under csrc/ or include/ is newer than the existing .so or it was compiled with other flags, the binding when its
source is newer or it was compiled against another torch or Python (its stamp, beside it, says which).
"""
from __future__ import annotations

import json
import os
import subprocess
import sys
import sysconfig
import time

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libtq.so")
BIND = os.path.join(PKG, "_bind.so")
BIND_SOURCE = "tq_bind.cpp"
BIND_STAMP = os.path.join(PKG, "_bind.stamp")           # what the binding was compiled against
BUILD_DIR = os.path.join(PKG, "_build")
LIB_FLAGS = os.path.join(BUILD_DIR, "libtq.flags")       # extra flags of the library (unknown if the file is not there)

ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _sources():
    out = []
    for d in (CSRC, INCLUDE):
        for name in sorted(os.listdir(d)):
            if name.endswith((".cu", ".cuh", ".cpp", ".h")):
                out.append(os.path.join(d, name))
    return out


def _read(path: str) -> str | None:
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def _write(path: str, text: str) -> None:
    with open(path, "w") as f:
        f.write(text)


def _newer(path: str, sources) -> bool:
    """Whether a file is there and no source is newer."""
    return os.path.exists(path) and all(os.path.getmtime(s) <= os.path.getmtime(path) for s in sources)


def _bind_needs() -> str:
    """What a binding is tied to: the torch it is compiled against, its C++ ABI, and Python's."""
    import torch

    return json.dumps(dict(torch=torch.__version__, cxx11_abi=bool(torch._C._GLIBCXX_USE_CXX11_ABI),
                           python=sysconfig.get_config_var("SOABI")))


def _lib_current(extra=()) -> bool:
    flags = _read(LIB_FLAGS)
    return (_newer(LIB, [s for s in _sources() if os.path.basename(s) != BIND_SOURCE]) and
            (flags == json.dumps(list(extra)) or (flags is None and not extra)))


def _bind_current() -> bool:
    return (_newer(BIND, [os.path.join(CSRC, BIND_SOURCE), os.path.join(INCLUDE, "tq.h")]) and
            _read(BIND_STAMP) == _bind_needs())


def needs_build() -> bool:
    return not (_lib_current() and _bind_current())


# source -> (its kind, the files under csrc/ it is compiled from besides tq.h and tq_internal.h)
UNITS = {
    "tq_lib.cu": ("cu", ("tq_device.cuh", "tq_codec_kernels.cuh", "tq_attend_kernel.cuh", "tq_qjl_kernel.cuh")),
    "tq_pages.cu": ("cu", ("tq_device.cuh", "tq_pages_kernels.cuh")),
    "tq_host.cpp": ("cpp", ()),
}


def _fresh(obj: str, src: str, cmd) -> bool:
    """Whether an object file was compiled by this command and is newer than everything it is compiled from."""
    if not os.path.exists(obj) or _read(obj + ".cmd") != json.dumps(cmd):
        return False
    deps = [os.path.join(CSRC, n) for n in (src, "tq_internal.h", *UNITS[src][1])] + [os.path.join(INCLUDE, "tq.h")]
    return all(os.path.getmtime(d) < os.path.getmtime(obj) for d in deps)


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _build_bind(verbose: bool) -> None:
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           f"-I{sysconfig.get_paths()['include']}", "-I/usr/local/cuda/include", os.path.join(CSRC, BIND_SOURCE), "-o",
           BIND + ".tmp", f"-L{PKG}", "-l:libtq.so", "-Wl,-rpath,$ORIGIN", f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python"]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if verbose or r.returncode:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout)
    if r.returncode:
        raise RuntimeError("compiling tq_bind.cpp failed")
    os.replace(BIND + ".tmp", BIND)
    _write(BIND_STAMP, _bind_needs())


def _build_lib(force: bool, verbose: bool, extra) -> None:
    os.makedirs(BUILD_DIR, exist_ok=True)
    common = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", f"-I{INCLUDE}"]
    objs = []
    cmds = []
    for src, (kind, _) in UNITS.items():
        obj = os.path.join(BUILD_DIR, src + ".o")
        objs.append(obj)
        if kind == "cu":
            cmd = [nvcc(), *ARCH_FLAGS, *common, "-Xptxas", "-warn-spills", *extra, "-c",
                   os.path.join(CSRC, src), "-o", obj]
        else:
            cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-ffp-contract=off", f"-I{INCLUDE}",
                   "-I/usr/local/cuda/include", "-c", os.path.join(CSRC, src), "-o", obj]
        if force or not _fresh(obj, src, cmd):
            cmds.append((obj, cmd))
    procs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for _, c in cmds]
    for (obj, c), p in zip(cmds, procs):
        out, _ = p.communicate()
        if verbose or p.returncode:
            sys.stderr.write(" ".join(c) + "\n" + out)
        if p.returncode:
            raise RuntimeError(f"compilation failed: {' '.join(c[:2])} ...")
        _write(obj + ".cmd", json.dumps(c))
    tmp = LIB + ".tmp"
    link = [nvcc(), *ARCH_FLAGS, "-shared", "-o", tmp, *objs, "-lcudart_static", "-lrt", "-lpthread", "-ldl"]
    r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode:
        sys.stderr.write(" ".join(link) + "\n" + r.stdout)
        raise RuntimeError("link failed")
    os.replace(tmp, LIB)
    _write(LIB_FLAGS, json.dumps(list(extra)))


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    t0 = time.time()
    lib, bind = force or not _lib_current(extra), force or not _bind_current()
    if lib:
        _build_lib(force, verbose, extra)
    if bind:
        _build_bind(verbose)
    if verbose and (lib or bind):
        sys.stderr.write(f"built {LIB if lib else BIND} in {time.time() - t0:.1f}s\n")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
