"""Plans of the norm and rotation of queries and keys, walked on the host."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_element_of_every_head_is_counted_once(tmp_path):
    """All D in 1..1024 and even R, both types: the program walks the kernels' own plans."""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")
    exe = str(tmp_path / "walk")
    build = subprocess.run([cxx, "-std=c++17", "-O2", "-Wno-unknown-pragmas", "-D__host__=", "-D__device__=", "-D__forceinline__=inline",
                            "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "state_space_sequence_ssm_amd", "csrc"),
                            os.path.join(ROOT, "tests", "rope_plan_walk.cpp"), "-o", exe], capture_output=True, text=True)
    assert build.returncode == 0, build.stderr[-2000:]
    run = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout
