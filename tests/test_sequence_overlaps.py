"""The sequence operators' overlap checks against the tensors' exact bytes (CPU only): sequence.cpp built with g++ under
AddressSanitizer and UndefinedBehaviorSanitizer, its launchers replaced by ones that lay out every run of bytes a
call reads and writes (tests/sanitize/sequence_overlaps.cpp)."""
import os
import shutil
import subprocess

import pytest

from test_sequence_sanitizers import CSRC, ROOT, SAN


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_accepted_calls_write_where_nothing_else_is(tmp_path):
    exe = str(tmp_path / "overlaps")
    cmd = ["g++", "-std=c++17", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include", "-I" + CSRC, "-I" + os.path.join(ROOT, "include"),
           os.path.join(CSRC, "sequence.cpp"), os.path.join(ROOT, "tests", "sanitize", "sequence_overlaps.cpp"), "-o", exe] + SAN + \
          ["-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe, "40000"], capture_output=True, text=True, env=env, timeout=300)
    assert r.returncode == 0 and "failed checks 0" in r.stdout, r.stdout[-2000:] + r.stderr[-4000:]
