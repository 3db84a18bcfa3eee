"""Build libtpla.so in-tree with nvcc for sm_100a, and beside it the Python
extension that marshals the tpla_kv_* calls.

The library is C and needs nvcc alone.  The extension needs torch with CUDA,
g++ and Python's headers, and belongs to the Python and torch it was built
with: both are in its name, so that others look for one of their own.

Usage: python -m mla_latent_kv_dim_b200.build [--force]
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libtpla.so")
SOURCES = ["api.cu", "decode_generic.cu", "decode_sm100.cu", "merge.cu", "hadamard.cu",
           "vup.cu", "noalloc.cu", "pca.cu", "append.cu", "kv_api.cu", "kv_append.cu", "kv_decode.cu",
           "kv_prefill.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _flags() -> list[str]:
    return ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                   "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
                   "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def binding_path() -> str:
    """The extension of this Python and torch."""
    import torch
    return os.path.join(PKG, f"_kvbind.torch-{torch.__version__}"
                             f"{sysconfig.get_config_var('EXT_SUFFIX')}")


def _binding_command(target: str) -> list[str]:
    """g++ command of the extension (torch's headers and libraries; no CUDA
    code)."""
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", os.path.join(ROOT, "include"), "-isystem", sysconfig.get_paths()["include"],
            "-isystem", os.path.join(base, "include"),
            "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(cuda, "include"),
            os.path.join(CSRC, "kv_binding.cpp"), "-o", target,
            "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _run(cmd: list[str], verbose: bool) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("compiler failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr)


def build(force: bool = False, verbose: bool = False) -> str:
    """The library; returns its path."""
    os.makedirs(OBJ, exist_ok=True)
    nvcc = _nvcc()
    headers = [os.path.join(ROOT, "include", "tpla.h")] + [
        os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OBJ, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([nvcc, *_flags(), "-c", s, "-o", o])
    with ThreadPoolExecutor(max_workers=min(8, max(1, len(jobs)))) as ex:
        list(ex.map(lambda cmd: _run(cmd, verbose), jobs))
    if force or jobs or _stale(LIB, objs):
        _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", LIB, *objs,
              "-Xlinker", "--no-undefined", "-ldl"], verbose)
    return LIB


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """The extension; returns its path."""
    target = binding_path()
    if force or _stale(target, [os.path.join(CSRC, "kv_binding.cpp"),
                                os.path.join(ROOT, "include", "tpla.h")]):
        # under another name until it is whole: other processes may look for it
        part = f"{target}.{os.getpid()}"
        try:
            _run(_binding_command(part), verbose)
            os.replace(part, target)
        finally:
            if os.path.exists(part):
                os.remove(part)
    return target


def main() -> int:
    force = "--force" in sys.argv
    print(build(force=force, verbose=True))
    try:
        print(build_binding(force=force, verbose=True))
    except (ImportError, OSError, RuntimeError) as e:
        print(f"The library is built. Python's kv_append, kv_decode and kv_prefill need an "
              f"extension that could not be built here:\n{e}", file=sys.stderr)
    return 0


if __name__ == "__main__":
    sys.exit(main())
