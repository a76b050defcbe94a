"""The build of a tree that holds sources alone, in processes of their own."""

import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "combine_moe_dispatch_layout_amd"


def run(code, where, env=None):
    return subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=where,
                          timeout=600, env={**os.environ, **(env or {})})


@pytest.fixture
def sources(tmp_path):
    """A copy of what a clone has: no built files."""
    built = shutil.ignore_patterns("*.so", "*.o", "_build", "__pycache__")
    for folder in (PACKAGE, "include", "oracle", "workloads"):
        shutil.copytree(os.path.join(ROOT, folder), tmp_path / folder, ignore=built)
    shutil.copy(os.path.join(ROOT, "__graft_entry__.py"), tmp_path)
    return tmp_path


def test_sources_alone_build_and_load_in_one_process(sources):
    """build() imports the package before there is anything to load; what it
    makes is found all the same, by the fast calls too."""
    out = run("import __graft_entry__ as g\n"
              "g.build()\n"
              "import torch, combine_moe_dispatch_layout_amd as m\n"
              "t = torch.zeros((3, 8))\n"
              "assert m._matrix_facts(t, torch.float32) == (-1, 3, 8, 8, t.data_ptr())\n"
              "lib = m.load_library()\n"
              "assert lib.moe_route is m._binding.moe_route\n"
              "assert m._binding.moe_route(None, 2, 8, None, 0, 8, 2, 0, 1, 1, 0, 1, 1.0, None,\n"
              "                            None, None) == m.MOE_OK\n"
              "print('from', m.__file__)\n", sources)
    assert out.returncode == 0, out.stdout + out.stderr
    assert f"from {sources}" in out.stdout


def test_the_extension_counts_arguments_before_it_is_bound():
    out = run("import combine_moe_dispatch_layout_amd as m\n"
              "try:\n"
              "    m._binding.moe_route(1, 2)\n"
              "except TypeError as e:\n"
              "    print('raised:', e)\n", ROOT)
    assert "raised: moe_route takes 16 arguments" in out.stdout, out.stdout + out.stderr


@pytest.mark.parametrize("left", ["none", "one that cannot be loaded"])
def test_the_library_loads_without_the_extension(sources, left):
    """What does not use the extension works without it; what does says what is
    wrong with it."""
    shutil.copy(os.path.join(ROOT, PACKAGE, "libmoe_dispatch.so"), sources / PACKAGE)
    if left != "none":
        name = "_binding" + sysconfig.get_config_var("EXT_SUFFIX")
        (sources / PACKAGE / name).write_bytes(b"no shared object")
    out = run("import torch, combine_moe_dispatch_layout_amd as m\n"
              "assert m.load_library().moe_abi_version() > 0\n"
              "assert m.moe_dispatch_capacity(4, 2, 8, 128) == 8 * 128\n"
              "assert m.moe_router_logits_workspace_size(1, 64, 8) == 0\n"
              "x = torch.zeros((3, 64), dtype=torch.bfloat16)\n"
              "for call in (lambda: m.moe_rms_norm(x, x[0]), lambda: m.moe_route(x, 2),\n"
              "             lambda: m.moe_router_logits(x, x)):\n"
              "    try:\n"
              "        call()\n"
              "    except ImportError as e:\n"
              "        print('raised:', e)\n", sources)
    assert out.returncode == 0, out.stderr
    said = "is missing: build it" if left == "none" else name
    lines = out.stdout.splitlines()
    assert len(lines) == 3 and all("raised:" in x and said in x for x in lines), out.stdout


def test_the_library_is_linked_whether_or_not_the_extension_compiles(sources):
    """A user of the C ABI needs no C++ compiler that knows Python and torch;
    that the extension was not made is an error all the same.  (A stand-in for
    hipcc writes the file it is asked for.)"""
    hipcc = sources / "hipcc"
    hipcc.write_text("#!/bin/sh\n"
                     "while [ \"$1\" != -o ]; do shift; done\n"
                     "echo made > \"$2\"\n")
    hipcc.chmod(0o755)
    out = run("from combine_moe_dispatch_layout_amd import build\n"
              "build.build()\n", sources,
              {"HIPCC": str(hipcc), "CXX": str(sources / "no-such-compiler")})
    assert out.returncode != 0 and "no-such-compiler" in out.stderr, out.stderr
    assert (sources / PACKAGE / "libmoe_dispatch.so").read_text() == "made\n"
