"""Build libsagesla.so in-tree with nvcc for sm_100a (B200).

python -m sparse_bit_attention_smoothing_b200.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libsagesla.so")
LAYER_DIR = PKG  # the compiled part of the Python binding (csrc/binding.cpp): _layer-<what it was compiled against>.so
SOURCES = ["k_prologue.cu", "k_topk.cu", "k_linear.cu", "k_flash.cu", "k_flash64.cu", "k_watchdog.cu", "k_w8a8.cu", "k_w8a8_token.cu", "k_qk_norm_rope.cu",
           "k_linear_decay.cu", "api.cu", "noalloc.cu"]
HEADERS = ["common.cuh", "kernels.h", "tensormap.h"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "-diag-suppress", "177"]
LAYER_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-shared", "-w", "-DTORCH_EXTENSION_NAME=_layer", "-DTORCH_API_INCLUDE_EXTENSION_H"]


def _nvcc() -> str:
    n = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(n):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsagesla.so")
    return n


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "sagesla.h")]
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            jobs.append([nvcc, *ARCH, *FLAGS, "-I", os.path.join(ROOT, "include"), "-c", s, "-o", o])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        list(ex.map(run, jobs))
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp%d" % os.getpid()
        run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"])
        os.replace(tmp, LIB)
    build_layer(force)
    return LIB


def layer_path() -> str | None:
    """The compiled binding for the torch (its version and where its libraries are), the Python ABI and the flags of now: they
    are in the file's name, so one that was compiled against others is neither taken for it nor loaded.  None where torch
    is not installed.  (torch is not imported for it.)"""
    import hashlib
    import importlib.metadata
    import importlib.util
    import sysconfig
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return None
    key = [importlib.metadata.version("torch"), os.path.dirname(spec.origin), sysconfig.get_config_var("SOABI"), *LAYER_FLAGS]
    return os.path.join(LAYER_DIR, "_layer-%s.so" % hashlib.sha256("\n".join(key).encode()).hexdigest()[:12])


def build_layer(force: bool = False) -> str | None:
    """The compiled binding of the layer operators, against the installed torch and libsagesla.so.  Without torch there is
    nothing to bind to and nothing is built: the C library needs nvcc alone."""
    layer = layer_path()
    if layer is None:
        return None
    src = os.path.join(CSRC, "binding.cpp")
    if not force and not _stale(layer, [src, os.path.join(ROOT, "include", "sagesla.h")]):
        return layer
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ext
    inc = [f"-I{p}" for p in ext.include_paths("cuda") + [sysconfig.get_paths()["include"]]]
    libs = [a for p in ext.library_paths("cuda") for a in (f"-L{p}", f"-Wl,-rpath,{p}")]
    tmp = layer + ".tmp%d" % os.getpid()
    cmd = [shutil.which("g++") or "g++", *LAYER_FLAGS, f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *inc,
           src, "-o", tmp, f"-L{PKG}", "-lsagesla", "-Wl,-rpath,$ORIGIN", *libs, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    for f in os.listdir(LAYER_DIR):  # those for another torch, Python or flags
        if f.startswith("_layer") and f.endswith(".so"):
            os.remove(os.path.join(LAYER_DIR, f))
    os.replace(tmp, layer)
    return layer


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
