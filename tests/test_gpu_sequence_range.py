"""The sequence operators at the ends of their sizes: rows of 2^31 - 1 positions and channels whose states pass 2^31
values, each compared bit for bit with calls on pieces of the same data."""
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


def test_conv_step_of_the_most_channels():
    """More than 2^31 values of state in one sequence."""
    g, K = _gen(5), 8
    D, n = (1 << 31) // (K - 1) + 1001, 4096
    x, w = torch.ones(1, D, dtype=torch.bfloat16, device="cuda"), torch.full((D, K), 0.25, device="cuda")
    state = torch.ones(1, D, K - 1, dtype=torch.bfloat16, device="cuda")
    ends = [slice(0, n), slice(D // 2, D // 2 + n), slice(D - n, D)]
    for s in ends:
        x[:, s], w[s], state[:, s] = _randn(g, 1, n, dtype=x.dtype), _randn(g, n, K), _randn(g, 1, n, K - 1, dtype=x.dtype)
    parts = [(x[:, s].clone(), state[:, s].clone(), w[s].clone()) for s in ends]
    out = sc.causal_conv_step(x, state, w, silu=False)
    for s, (px, ps, pw) in zip(ends, parts):
        assert torch.equal(out[:, s], sc.causal_conv_step(px, ps, pw, silu=False)) and torch.equal(state[:, s], ps)
    assert (out[:, n:D // 2] == 2).all() and (out[:, D // 2 + n:D - n] == 2).all()
