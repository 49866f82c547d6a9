"""Build libbiloco.so (sm_100a) in-tree with nvcc, and the Python fast path beside it.

    python -m nvfp4_binary_rank_b200.build          # incremental
    python -m nvfp4_binary_rank_b200.build --force  # rebuild

Every .cu file under csrc/ is compiled to an object in parallel (the fused
kernel instances live in separate files for that reason), then linked.  The
library links the CUDA runtime dynamically so that, inside a process that
already imported PyTorch, it shares PyTorch's runtime (one current device, one
context).  Nothing here needs a GPU.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libbiloco.so")
BINDING = os.path.join(PKG, "_binding.so")
OBJ = os.path.join(PKG, "_build")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + [os.path.join(INCLUDE, "biloco.h")])


def _obj_of(src):
    return os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")


def _compile(src, force, verbose):
    obj = _obj_of(src)
    newest_dep = max(os.path.getmtime(p) for p in _headers() + [src])
    if not force and os.path.exists(obj) and os.path.getmtime(obj) >= newest_dep:
        return obj
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}")
    os.replace(obj + ".tmp", obj)
    return obj


def _build_binding(force, verbose):
    """The FP8 operators' fast Python path (csrc/binding.cpp), against PyTorch's headers."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    src, stamp = os.path.join(CSRC, "binding.cpp"), os.path.join(OBJ, "binding.torch")
    newest = max(os.path.getmtime(p) for p in (src, os.path.join(INCLUDE, "biloco.h")))
    built_for = open(stamp).read() if os.path.exists(stamp) else None
    if not force and os.path.exists(BINDING) and os.path.getmtime(BINDING) >= newest and built_for == torch.__version__:
        return
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DBILOCO_TORCH_VERSION="{torch.__version__}"',
           *(f"-I{p}" for p in [*cpp_extension.include_paths(), cuda, sysconfig.get_paths()["include"]]),
           src, "-o", BINDING + ".tmp", f"-L{PKG}", "-l:libbiloco.so", "-Wl,-rpath,$ORIGIN",
           *(f"-L{p}" for p in cpp_extension.library_paths()), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
           "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("the compiler failed on binding.cpp")
    os.replace(BINDING + ".tmp", BINDING)
    with open(stamp, "w") as f:
        f.write(torch.__version__)


def build(force: bool = False, verbose: bool = False) -> str:
    lib = _build_library(force, verbose)
    try:
        _build_binding(force, verbose)
    except (RuntimeError, OSError) as e:
        # the library serves every call without it; an older one may not match the library any more
        if os.path.exists(BINDING):
            os.remove(BINDING)
        sys.stderr.write(f"built without the FP8 calls' fast path: {e}\n")
    return lib


def _build_library(force, verbose) -> str:
    os.makedirs(OBJ, exist_ok=True)
    srcs = sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(lambda s: _compile(s, force, verbose), srcs))
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= max(os.path.getmtime(o) for o in objs):
        return LIB
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "shared", "-o", LIB + ".tmp", *objs,
           "-Xlinker", "-rpath,/usr/local/cuda/lib64"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("nvcc failed linking libbiloco.so")
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
