"""Builds libmoe_gb300.so (the C-ABI library) with nvcc for sm_103a.

Each .cu file is compiled in its own nvcc process (in parallel), then linked
into one shared library with the CUDA runtime linked statically, so the library
loads on a machine without a GPU (calls then fail with MOE_ERR_CUDA).  Beside it,
where PyTorch is installed, _ops.so: the Python entries of the operators around the
layer, against its headers.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoe_gb300.so")
SOURCES = ["gemm.cu", "api.cu", "gate.cu", "align.cu", "route.cu", "reduce.cu", "noalloc.cu", "scale.cu",
           "repack.cu", "ops_api.cu", "norm.cu", "router.cu", "fp8_block.cu", "fp8_few.cu", "few.cu"]
OPS = os.path.join(PKG, "_ops.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(obj: str, deps: list[str]) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def _torch_version() -> str | None:
    """Of the installed PyTorch, None without one."""
    if importlib.util.find_spec("torch") is None:
        return None
    return importlib.metadata.version("torch")


def _ops_command(obj: str) -> list[str]:
    import sysconfig
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    include = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[f"-isystem{i}" for i in include], "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]


def _link_ops(obj: str) -> list[str]:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++", "-shared", "-o", OPS, obj, LIB, "-Wl,-rpath,$ORIGIN", "-L" + lib, "-ltorch_python", "-ltorch_cpu",
            "-lc10_cuda", "-lc10"]


def _start(cmd: list[str], verbose: bool) -> subprocess.Popen:
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _finish(procs: list[tuple[str, subprocess.Popen]], verbose: bool) -> None:
    failed = []
    for src, pr in procs:
        out, _ = pr.communicate()
        text = out.decode(errors="replace")
        if pr.returncode != 0:
            failed.append(f"--- {src}\n{text}")
        elif verbose and text.strip():
            print(text, flush=True)
    if failed:
        raise RuntimeError("build failed:\n" + "\n".join(failed))


def build(verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    headers = [os.path.join(CSRC, h) for h in os.listdir(CSRC) if h.endswith((".h", ".cuh"))]
    headers.append(os.path.join(ROOT, "include", "moe.h"))
    procs, objs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if _stale(o, [s] + headers):
            procs.append((src, _start([cc, *ARCH, *FLAGS, *(extra_flags or []), "-c", s, "-o", o], verbose)))
    # The Python entries need PyTorch and fit the one (and the Python) whose headers they saw; the library needs neither.
    torch_version = _torch_version()
    ops_obj = os.path.join(BUILD, f"binding-{torch_version}-{sys.implementation.cache_tag}.o")
    ops_procs = []
    if torch_version is not None and _stale(ops_obj, [os.path.join(CSRC, "binding.cpp"), headers[-1]]):
        ops_procs.append(("binding.cpp", _start(_ops_command(ops_obj), verbose)))
    try:
        _finish(procs, verbose)
        if _stale(LIB, objs):
            _finish([(LIB, _start([cc, *ARCH, "-shared", "-Xlinker", "-soname=libmoe_gb300.so", "-o", LIB, *objs, "-cudart",
                                   "static"], verbose))], verbose)
    finally:
        _finish(ops_procs, verbose)
    if torch_version is None:
        print(f"no PyTorch: {os.path.basename(OPS)} is not built", file=sys.stderr)
        return LIB
    stamp = os.path.join(BUILD, "_ops.for")
    fits = os.path.exists(stamp) and open(stamp).read() == os.path.basename(ops_obj)
    if not fits or _stale(OPS, [ops_obj, LIB]):
        _finish([(OPS, _start(_link_ops(ops_obj), verbose))], verbose)
        with open(stamp, "w") as f:
            f.write(os.path.basename(ops_obj))
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
