"""Caps far above the scores: cap tanh(s / cap) is then nearly s itself, and the outputs those without a cap.

Tolerance: the bound of the call without a cap (tests/attention_ref.py), and what the cap adds to a score's error, E: s - cap tanh(s / cap) is at
most |s|^3 / (3 cap^2); the kernels' tanh is off by 4 U of itself in fp32, in 16-bit types by 2^-22 of 1 under caps up to 1024 and by 2^-19 of
itself above; its argument and the product with the cap by 4 U more.  Weights off by E relative move an output by at most
E (sum p |v| / sum p + |out|) <= 2 E max |v|, 5% for the second order."""
import pytest
import torch

import attention_ref as ref
import sparse_weight_direct_amd as sc
from test_gpu_attention import INF, NAN, TYPES, _cache, _gen, _ints, _randn

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _check(g, dtype, D, L, past, cap, change=None, **kw):
    k, v, table = _cache(g, dtype, 2, D, 32, past, None, L)
    q = _randn(g, 2, 6 * D, L, dtype=dtype, scale=3.0)
    kk = torch.nan_to_num(ref.wide(k))
    largest = float(torch.nan_to_num(ref.wide(v)).abs().max())
    if change:
        change(v, table)
    out, bound, finite = ref.paged_attention(q, k, v, table, _ints(past), out_dtype=torch.float32, **kw)
    keys = kk.permute(1, 3, 0, 2).reshape(2, D, -1)  # (G, D, all positions)
    s = max(float((ref.wide(q)[:, h * D:(h + 1) * D].transpose(1, 2) @ keys[h // 3]).abs().max()) for h in range(6)) * D ** -0.5
    E = s ** 3 / (3 * cap ** 2) + 4 * U * s
    E += 4 * U * s if dtype == torch.float32 else cap * 2.0 ** -22 if cap <= 1024 else s * 2.0 ** -19
    got = torch.full(q.shape, NAN, device="cuda")
    sc.paged_attention(q, k, v, table, _ints(past), cap=cap, out=got, **{n: _ints(t) if n == "prefix" else t for n, t in kw.items()})
    ref.check_attention(got, (out, bound + 1.05 * 2 * E * largest, finite), f"{dtype} {D} {L} {cap}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [1, 6, 40, 150])
@pytest.mark.parametrize("cap", [300.0, 1024.0, 1025.0, 1e5, 1e7, 1e30])
def test_caps_far_above_the_scores(dtype, L, cap):
    _check(_gen(L), dtype, 64, L, [17, 200], cap)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [40, 80, 128, 200, 256])
@pytest.mark.parametrize("L", [1, 4, 40, 150])
def test_every_width(dtype, D, L):
    _check(_gen(D), dtype, D, L, [0, 90], 3e6)
    _check(_gen(D), dtype, D, L, [2000, 5], 3e6, window=80, prefix=[10, 3])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("L", [3, 40, 150])
def test_infinities_in_part_of_the_rows(dtype, D, L):
    def change(v, table):
        v[int(table[0, 1]), 0, 3, 5], v[int(table[0, 1]), 1, 7, 4] = INF, NAN

    _check(_gen(D), dtype, D, L, [36, 36], 3e6, change=change)
    _check(_gen(D), dtype, D, L, [36, 36], 3e6, change=change, window=2)
