"""How the attention operators' launches are cut (CPU only: csrc/attention_plan.h built with g++ under the sanitizers): what the documented
limits let through fits a launch, up to the ends of the sizes' types."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_weight_direct_amd", "csrc")
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer", "-g", "-O1"]


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_what_fits_is_a_launch(tmp_path):
    exe = str(tmp_path / "attention_plans")
    subprocess.run(["g++", "-std=c++17", "-I" + CSRC, "-I" + os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "sanitize", "attention_plans.cpp"), "-o", exe] + SAN, check=True)
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe, "300000"], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "failed checks 0" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
