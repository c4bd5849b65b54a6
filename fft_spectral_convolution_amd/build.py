"""Build libfno.so (HIP, gfx950) in-tree.

    python -m fft_spectral_convolution_amd.build      # or: python fft_spectral_convolution_amd/build.py

Compiles every csrc/*.hip for gfx950 with hipcc into objects under _build/
and links them into fft_spectral_convolution_amd/libfno.so; and, with the host
compiler, the reader of tensor lists for the Python binding (csrc/fno_lists.cpp)
into fft_spectral_convolution_amd/_fno_lists.so.  Always recompiles.  Packed-fp32 instruction selection is switched off for all device
code.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfno.so")
LISTS = os.path.join(PKG, "_fno_lists.so")

ARCH = "gfx950"
FLAGS = [
    "-O3",
    "-std=c++17",
    f"--offload-arch={ARCH}",
    "-fPIC",
    "-Wall",
    "-Wno-unused-function",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP toolchain is required to build libfno")


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [hipcc()] + FLAGS + ["-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    warn = "\n".join(l for l in res.stderr.splitlines() if "packed-fp32-ops" not in l and l.strip())
    if verbose and warn:
        print(warn, file=sys.stderr)
    return obj


def build_lists(verbose: bool = False) -> str:
    """The reader of tensor lists: host code against torch's and Python's headers."""
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = LISTS + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{p}" for p in include_paths()], f"-I{sysconfig.get_paths()['include']}",
           os.path.join(CSRC, "fno_lists.cpp"), "-o", tmp, f"-L{libs}", f"-Wl,-rpath,{libs}", "-ltorch_python",
           "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on fno_lists.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LISTS)
    return LISTS


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    # those of many template instances first: they take minutes, the others seconds
    sources = sorted(glob.glob(os.path.join(CSRC, "*.hip")),
                     key=lambda s: (not os.path.basename(s).startswith(("fno_channels_", "fno_groupnorm")), s))
    if not sources:
        raise RuntimeError(f"no HIP sources under {CSRC}")
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(sources))) as ex:
        lists = ex.submit(build_lists, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), sources))
        lists.result()
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
