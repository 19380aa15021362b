"""Build libfa_sm100.so in-tree with nvcc for sm_100a, and the compiled part of
the Python binding with g++."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = [os.path.join(HERE, "csrc", "fa_api.cu"),
           os.path.join(HERE, "csrc", "fa_noalloc.cu"),
           os.path.join(HERE, "csrc", "fa_paged.cu"),
           os.path.join(HERE, "csrc", "fa_rope.cu")]


def headers():
    """Every header the sources can include: all of csrc/*.cuh, csrc/*.h and include/*.h."""
    out = []
    for folder in (os.path.join(HERE, "csrc"), os.path.join(ROOT, "include")):
        out += sorted(os.path.join(folder, f) for f in os.listdir(folder)
                      if f.endswith((".cuh", ".h")))
    return out

OUT = os.path.join(HERE, "libfa_sm100.so")
BINDING_SOURCE = os.path.join(HERE, "csrc", "fa_binding.cpp")


def nvcc_command(out: str = OUT, extra=()):
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return [nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo",
            "-std=c++17", "-Xcompiler", "-fPIC", "-shared",
            "-I", os.path.join(ROOT, "include"), "-o", out, *SOURCES, *extra]


def binding_path() -> str:
    """Where the compiled part of the Python binding is: its name holds the torch
    and the Python that it is built for, whose C++ and C interfaces it calls, so
    that under others it is built anew and not loaded."""
    import torch
    return os.path.join(HERE, f"_fa_binding.torch-{torch.__version__}"
                              f"{sysconfig.get_config_var('EXT_SUFFIX')}")


def binding_command(out: str):
    """The compiled part of the Python binding, against this torch's headers."""
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    flags = []
    for p in include_paths(device_type="cuda") + [sysconfig.get_paths()["include"]]:
        flags += ["-isystem", p]
    for p in library_paths(device_type="cuda"):
        flags += ["-L", p]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", os.path.join(ROOT, "include"), *flags, "-o", out, BINDING_SOURCE,
            "-L", HERE, "-l:" + os.path.basename(OUT), "-Wl,-rpath,$ORIGIN",
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python"]


def up_to_date(out: str = OUT, sources=None) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(f) <= t for f in (sources or SOURCES + headers()))


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not up_to_date():
        extra = ["-Xptxas", "-v"] if verbose else []
        subprocess.run(nvcc_command(extra=extra), check=True)
    binding = binding_path()
    if force or not up_to_date(binding, [BINDING_SOURCE, os.path.join(ROOT, "include", "fa.h")]):
        subprocess.run(binding_command(binding), check=True)
    return OUT


if __name__ == "__main__":
    build(force="--changed" not in sys.argv, verbose="-v" in sys.argv)
    print(OUT)
