"""Scores far from 0 and infinite ones in visible places, in every type, for few and for many rows; outputs held to tests/attention_ref.py."""
import pytest
import torch

import attention_ref as ref
import sparse_weight_direct_amd as sc
from test_gpu_attention import INF, TYPES, _cache, _check, _gen, _ints, _randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("L", [1, 3, 40, 150])
def test_scores_far_from_zero(dtype, D, L):
    """One row's scores are hundreds, of either sign; weights beside the largest are down to nothing (fp16: subnormal)."""
    g = _gen(L + D)

    def change(q, k, v, table):
        q[:, :, 0] *= 30.0
        q[:, :, -1] = -20.0

    for f32 in (False, True) if dtype != torch.float32 else (False,):
        _check(g, dtype, 1, 2, 1, D, L, 16, [20], change=change, spread=5.0, out_f32=f32)
        _check(g, dtype, 1, 4, 2, D, L, 64, [300], change=change, spread=2.0, out_f32=f32, window=70)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("L", [1, 5, 40, 150])
def test_a_score_of_minus_infinity_is_a_weight_of_zero(dtype, D, L):
    """A page of such keys, first in the context: the same as a page that is not there."""
    g = _gen(L)
    past = [40, 150]
    k, v, table = _cache(g, dtype, 2, D, 16, past, None, L)
    q = _randn(g, 2, 4 * D, L, dtype=dtype)
    q[:, ::D] = 1.0
    hidden = table.clone()
    hidden[:, 0] = -1
    want = ref.paged_attention(q, k, v, hidden, _ints(past))
    for b in range(2):
        k[int(table[b, 0]), :, :, 0] = -INF
    ref.check_attention(sc.paged_attention(q, k, v, table, _ints(past)), want)
    for b in range(2):  # in the middle, some of them, and one of plus infinity, which spoils the rows that see it
        k[int(table[b, 0]), :, :, 0] = 0.0
        k[int(table[b, 1]), :, 3:7, 0] = -INF
    assert torch.isfinite(sc.paged_attention(q, k, v, table, _ints(past))).all()
    k[int(table[1, 2]), 0, 5, 0] = INF
    got = sc.paged_attention(q, k, v, table, _ints(past)).view(2, 4, D, L)
    assert torch.isnan(got[1, :2]).all() and torch.isfinite(got[1, 2:]).all() and torch.isfinite(got[0]).all()
