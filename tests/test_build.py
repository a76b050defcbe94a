"""The build of a tree that holds sources alone, in processes of their own."""

import os
import shutil
import subprocess
import sys

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
