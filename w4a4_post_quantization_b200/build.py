"""Builds ``libkq.so`` in-tree with nvcc for sm_100a (no fast-math: IEEE
float32 with denormals is part of the quantizer's contract), and
``_kq_torch.so``, the compiled part of the Python binding."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
OUT = os.path.join(HERE, "libkq.so")
BINDING = os.path.join(HERE, "_kq_torch.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17", "--threads", "0",
    "-Xcompiler", "-fPIC", "-shared",
]


def sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cuh")) +
                  glob.glob(os.path.join(HERE, "csrc", "*.h")) +
                  glob.glob(os.path.join(ROOT, "include", "*.h")))


def binding_sources():
    return [os.path.join(HERE, "csrc", "kq_torch.cpp"), os.path.join(ROOT, "include", "kq.h")]


def _newer(out, files) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(f) <= t for f in files)


def up_to_date() -> bool:
    return _newer(OUT, sources() + headers() + [__file__]) and \
        _newer(BINDING, binding_sources() + [__file__])


def _cuda_include():
    """The headers beside nvcc, which may be a bare name or a link."""
    nvcc = os.path.realpath(shutil.which(NVCC) or NVCC)
    return os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")


def _binding_command():
    import torch
    from torch.utils import cpp_extension as ext
    includes = [*ext.include_paths(), _cuda_include(), sysconfig.get_paths()["include"],
                os.path.join(ROOT, "include")]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[a for i in dict.fromkeys(includes) for a in ("-isystem", i)],
            "-o", BINDING + ".tmp", binding_sources()[0], "-L", lib,
            "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda"]


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return OUT
    cmd = [NVCC, *FLAGS, "-I", os.path.join(ROOT, "include"), "-o", OUT + ".tmp", *sources()]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    binding = failure = None
    try:
        binding = subprocess.Popen(_binding_command())
    except Exception as e:                       # the library is built and installed all the same
        failure = e
    try:
        subprocess.run(cmd, check=True)
        os.replace(OUT + ".tmp", OUT)
    finally:
        status = binding.wait() if binding else None
    if failure:
        raise failure
    if status != 0:
        raise subprocess.CalledProcessError(status, binding.args)
    os.replace(BINDING + ".tmp", BINDING)
    return OUT


if __name__ == "__main__":
    print(build(force=True, verbose=True))
