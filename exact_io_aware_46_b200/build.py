"""Builds the CUDA library ``libattn.so`` (nvcc, sm_100a only) and the Python extension
``_binding`` (g++, against torch's headers) in-tree.  The library works without the extension, so
a failure to build that one is a warning."""

from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SO = os.path.join(HERE, "libattn.so")
SRC = os.path.join(HERE, "csrc", "attn_api.cu")
SRC_NOALLOC = os.path.join(HERE, "csrc", "decode_noalloc.cu")
BINDING = os.path.join(HERE, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
SRC_BINDING = os.path.join(HERE, "csrc", "binding.cpp")


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    return "nvcc"


def sources():
    return [SRC, SRC_NOALLOC] + sorted(glob.glob(os.path.join(HERE, "csrc", "*.cuh"))) + [
        os.path.join(ROOT, "include", "attn.h")]


def up_to_date(so: str, srcs) -> bool:
    if not os.path.exists(so):
        return False
    t = os.path.getmtime(so)
    return all(os.path.getmtime(s) <= t for s in srcs)


def binding_up_to_date() -> bool:
    from . import BINDING_TAG

    if not up_to_date(BINDING, [SRC_BINDING, os.path.join(ROOT, "include", "attn.h")]):
        return False
    with open(BINDING, "rb") as f:  # the tag is a string of the extension
        return BINDING_TAG.encode() in f.read()


def build_binding(force: bool = False) -> str:
    if not force and binding_up_to_date():
        return BINDING
    import torch

    from . import BINDING_TAG

    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.sep in nvcc() else "/usr/local/cuda"
    inc = [os.path.join(ROOT, "include"), os.path.join(t, "include"),
           os.path.join(t, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = BINDING + f".tmp{os.getpid()}"
    subprocess.check_call(
        [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
         f'-DBINDING_TAG="{BINDING_TAG}"']
        + ["-I" + i for i in inc] + [SRC_BINDING, "-o", tmp, "-L" + os.path.join(t, "lib")]
        + ["-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10"])
    os.replace(tmp, BINDING)
    return BINDING


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date(SO, sources()):
        return SO
    tmp = SO + f".tmp{os.getpid()}"
    cmd = [nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3",
           "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I", os.path.join(ROOT, "include"),
           "-Xptxas", "-v" if verbose else "-O3", SRC, SRC_NOALLOC, "-o", tmp]
    subprocess.check_call(cmd)
    os.replace(tmp, SO)
    return SO


def build(force: bool = False, verbose: bool = False) -> str:
    so = build_library(force, verbose)
    try:
        build_binding(force)
    except (OSError, subprocess.CalledProcessError) as e:
        if os.path.exists(BINDING):  # of other sources or another torch
            os.remove(BINDING)
        warnings.warn(f"the Python extension was not built, its calls run in Python: {e}",
                      RuntimeWarning, stacklevel=2)
    return so


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
