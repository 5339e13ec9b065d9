"""The sequence operators at the ends of their sizes: rows of 2^31 - 1 positions, compared bit for bit with calls
on pieces of the same data."""
import pytest
import torch

import sparse_weight_direct_amd as sc
from test_gpu_sequence import _gen, _ints, _randn

pytestmark = pytest.mark.gpu

NAN = float("nan")


def _filled(g, n, dtype):
    """n random values, made of one random stretch whose length no power of two divides."""
    t, part = torch.empty(n, dtype=dtype, device="cuda"), _randn(g, (1 << 24) + 77, dtype=dtype)
    for at in range(0, n, part.numel()):
        t[at:at + part.numel()] = part[:n - at]
    return t


@pytest.mark.parametrize("L", [(1 << 31) - 1, (1 << 31) - 7])
def test_conv_longest_row(L):
    g, K = _gen(L), 4
    x, w, b = _filled(g, L, torch.bfloat16).view(1, 1, L), _randn(g, 1, K), _randn(g, 1)
    out = torch.full((1, 1, L), NAN, dtype=torch.bfloat16, device="cuda")
    state = torch.empty(1, 1, K - 1, dtype=torch.bfloat16, device="cuda")
    sc.causal_conv(x, w, b, final_state=state, out=out)
    assert torch.equal(state[0, 0], x[0, 0, L - K + 1:])
    step = 1 << 28
    for at in range(0, L, step):  # and nowhere is out left as it was
        n = min(step, L - at)
        before = x[:, :, at - K + 1:at].contiguous() if at else torch.zeros_like(state)
        assert torch.equal(out[:, :, at:at + n], sc.causal_conv(x[:, :, at:at + n], w, b, initial_state=before))
    n = L - 9  # shorter than the row: what lies past it is 0
    sc.causal_conv(x, w, b, lengths=_ints([n]), final_state=state, out=out)
    assert torch.equal(state[0, 0], x[0, 0, n - K + 1:n]) and not out[0, 0, n:].any() and out[0, 0, n - 100:n].all()
