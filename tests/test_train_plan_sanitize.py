"""The planners of the gated block and of the cross entropy built on the CPU with
the address and undefined-behaviour sanitizers and driven over contractions of
no and few values (tests/sanitize/train_plan_checks.cpp)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tile_partitioned_dense_amd", "csrc")


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
@pytest.mark.parametrize("opt", ["-O0", "-O2"])
def test_train_plans_under_asan_and_ubsan(tmp_path, opt):
    exe = str(tmp_path / "train_plan_checks")
    cmd = ["g++", "-std=c++17", opt, "-g", "-fno-omit-frame-pointer",
           "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC,
           os.path.join(ROOT, "tests", "sanitize", "train_plan_checks.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert r.stdout.startswith("ok ") and "runtime error" not in r.stderr, r.stdout + r.stderr
