"""The split of chunk attention over CTAs, as the kernels compile it, run on the CPU (walk_check.cpp): every
iteration of every unit by one CTA, what a CTA leaves for the join in one slot each, bad descriptions refused."""
import os
import subprocess

import pytest

from latency_moe_decode_persistent_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_split_covers_every_iteration_once(tmp_path):
    cuda = os.path.join(os.path.dirname(os.path.dirname(build._nvcc())), "include")
    if not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        pytest.skip("no CUDA headers beside nvcc")
    exe = str(tmp_path / "walk_check")
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", build.CSRC, "-I", cuda, os.path.join(ROOT, "tests", "walk_check.cpp"), "-o", exe],
                   check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.endswith("ok\n"), r.stdout[-2000:] + r.stderr[-2000:]
