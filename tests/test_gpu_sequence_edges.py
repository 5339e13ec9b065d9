"""The sequence operators at the ends of their values and arguments: infinite, extreme and absent
values in places where a result is still defined, and calls that must be refused before anything is
written.  Bounds are those of tests/sequence_ref.py unless a test states its own."""
import numpy as np
import pytest
import torch

import sequence_ref as ref
import sparse_weight_direct_amd as sc
from test_gpu_sequence import TYPES, _gen, _ints, _randn, _scan_inputs

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


# ---- states beside the last whole four


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 15, 18, 33])
def test_scan_step_infinite_input_at_any_state_size(dtype, N):
    """An infinite input with c = b and D > 0 makes every term infinite with its sign: so is the output, whatever
    N leaves of a lane's four states."""
    g = _gen(N)
    B, D = 3, 21
    x, dt = _randn(g, B, D, dtype=dtype), _randn(g, B, D, dtype=dtype)
    A, b, skip = -torch.exp(_randn(g, D, N)), _randn(g, B, 1, N, dtype=dtype), torch.ones(D, device="cuda")
    x[0, 4], x[2, 20] = INF, -INF
    state = _randn(g, B, D, N)
    out = sc.selective_scan_step(x, state, dt, A, b, b, D=skip)
    assert out[0, 4].item() == INF and out[2, 20].item() == -INF
    assert torch.equal(state[0, 4], b[0, 0].float().sign() * INF) and torch.equal(state[2, 20], b[2, 0].float().sign() * -INF)
    out[0, 4], out[2, 20] = 0.0, 0.0
    assert torch.isfinite(out).all()
