"""Build libmoe_dispatch.so (the HIP kernels + C ABI) for gfx950, and the
binding's C extension, in-tree.

    python -m combine_moe_dispatch_layout_amd.build

Each source is compiled to an object in parallel, then linked into one shared
library next to this file.  Flags: -O3, gfx950 only, and packed-fp32 code
generation disabled (the kernels' fp32 arithmetic is scalar by design).
"""

from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libmoe_dispatch.so")
SOURCES = ["api.hip", "layout.hip", "dispatch.hip", "fused.hip", "combine.hip", "backward.hip",
           "experts.hip", "norm.hip", "router.hip", "route.hip", "probe.hip", "noalloc.hip",
           "planner.cpp"]
ARCH = "gfx950"
# The Python binding's hot path (csrc/binding.cpp), for the interpreter that builds it.
BINDING = os.path.join(HERE, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
COMMON = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    "-Wno-unused-command-line-argument",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _obj_dir() -> str:
    d = os.path.join(HERE, "_build")
    os.makedirs(d, exist_ok=True)
    return d


# Build-time tuning macros (for example "-DMOE_CACHED_ROWS_PER_CU=8"); the
# defaults in csrc/moe_internal.h are the measured choices.
EXTRA = os.environ.get("MOE_HIPCC_DEFINES", "").split()


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(_obj_dir(), os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *COMMON, *EXTRA, f"-I{INCLUDE}", "-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    return obj


def _build_binding(verbose: bool) -> None:
    from torch.utils import cpp_extension
    import torch
    tmp = BINDING + f".tmp{os.getpid()}"
    includes = [f"-I{d}" for d in (INCLUDE, sysconfig.get_paths()["include"],
                                   *cpp_extension.include_paths())]
    libs = [f"-L{d}" for d in cpp_extension.library_paths()]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-Wall", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *includes,
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, *libs, "-lc10", "-ltorch_cpu",
           "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)


def _link(objs: list, verbose: bool) -> None:
    tmp = LIB + f".tmp{os.getpid()}"
    exports = os.path.join(CSRC, "exports.map")  # only the moe_* C ABI is exported
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC",
           f"-Wl,--version-script={exports}", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)


def build(verbose: bool = False) -> str:
    """Compile every source, link the shared library and the binding's
    extension; returns the library's path."""
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as pool:
        binding = pool.submit(_build_binding, verbose)
        objs = list(pool.map(lambda s: _compile(s, verbose), SOURCES))
        _link(objs, verbose)  # before the extension is asked for: the C ABI needs none
        binding.result()
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
