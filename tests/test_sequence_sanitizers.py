"""The sequence operators' argument checks under AddressSanitizer and UndefinedBehaviorSanitizer (CPU
only): sequence.cpp built with g++, its launchers replaced, driven with seeded random argument
structures (sizes and strides up to the ends of their types, addresses misaligned, overlapping or
NULL).  Any sanitizer report, missing message or accepted call that the kernels could not run fails."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sparse_weight_direct_amd", "csrc")
SAN = ["-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-fno-omit-frame-pointer", "-g", "-O1"]


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_argument_checks_under_sanitizers(tmp_path):
    exe = str(tmp_path / "fuzz_sequence")
    cmd = ["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + CSRC, "-I" + os.path.join(ROOT, "include"),
           os.path.join(CSRC, "sequence.cpp"), os.path.join(ROOT, "tests", "sanitize", "fuzz_sequence.cpp"), "-o", exe] + SAN + \
          ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe, "20000"], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "failed checks 0" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
