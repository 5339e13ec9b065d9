"""The package without the sequence operators' native binding (CPU only): the sparse convolution and the functions
with the C names need libsparseconv.so alone, and the operators that need the binding say that it is missing."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "sparse_weight_direct_amd")

CODE = """
import numpy as np, torch
import sparse_weight_direct_amd as sc
import sparse_weight_direct_amd.ssm
h = sc.Handle.from_dense(np.ones((4, 3, 1, 1), np.float32), 1, 5, 1, 0, flags=sc.SC_PACK_HOST_ONLY)
assert h.info()["nnz"] == 12, h.info()
assert sc.selective_scan_workspace(torch.empty(1, 4, 64), torch.empty(4, 16), 1) == 0
x = torch.zeros(1, 4, 5)
for call in (lambda: sc.causal_conv(x, x), lambda: sc.causal_conv_step(x, x, x), lambda: sc.selective_scan(x, x, x, x, x),
             lambda: sc.selective_scan_step(x, x, x, x, x, x), lambda: sc.adapter_apply(x, x, x, x)):
    try:
        call()
    except ImportError as e:
        assert "_binding" in str(e) and "build" in str(e), e
    else:
        raise AssertionError("no ImportError")
print("fine")
"""


@pytest.mark.parametrize("binding", ["missing", "unfit"])
def test_package_without_the_binding(tmp_path, binding):
    to = tmp_path / "sparse_weight_direct_amd"
    to.mkdir()
    for f in os.listdir(PKG):
        if f.endswith(".py"):
            shutil.copy(os.path.join(PKG, f), to)
    os.symlink(os.path.join(PKG, "libsparseconv.so"), to / "libsparseconv.so")
    if binding == "unfit":
        (to / "_binding.so").write_bytes(b"")
    r = subprocess.run([sys.executable, "-c", CODE], cwd=tmp_path, capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, PYTHONPATH=str(tmp_path)))
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stdout + r.stderr
