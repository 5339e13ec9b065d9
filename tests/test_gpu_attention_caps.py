"""Caps far above the scores: cap tanh(s / cap) is then s itself, and the outputs are those without a cap.

Tolerance: the bound of the call without a cap (tests/attention_ref.py), and what the cap adds to a score's error, E: s - cap tanh(s / cap) is at
most |s|^3 / (3 cap^2); the kernels' tanh is off by 2^-19 of itself (fp32: 4 U), its argument and the product with the cap by 4 U more.
Weights off by E relative move an output by at most E (sum p |v| / sum p + |out|) <= 2 E max |v|, 5% for the second order."""
import pytest
import torch

import attention_ref as ref
import sparse_weight_direct_amd as sc
from test_gpu_attention import TYPES, _cache, _gen, _ints, _randn

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [1, 6, 40, 150])
@pytest.mark.parametrize("cap", [300.0, 2e3, 1e5, 1e7, 1e30])
def test_caps_far_above_the_scores(dtype, L, cap):
    g = _gen(L)
    D, past = 64, [17, 200]
    k, v, table = _cache(g, dtype, 2, D, 32, past, None, L)
    q = _randn(g, 2, 6 * D, L, dtype=dtype, scale=3.0)
    out, bound, finite = ref.paged_attention(q, k, v, table, _ints(past), out_dtype=torch.float32)
    kk, vv = (torch.nan_to_num(ref.wide(t)) for t in (k, v))
    keys = kk.permute(1, 3, 0, 2).reshape(2, D, -1)  # (G, D, all positions)
    s = max(float((ref.wide(q)[:, h * D:(h + 1) * D].transpose(1, 2) @ keys[h // 3]).abs().max()) for h in range(6)) * D ** -0.5
    E = s ** 3 / (3 * cap ** 2) + s * ((4 * U if dtype == torch.float32 else 2.0 ** -19) + 4 * U)
    got = torch.full(q.shape, float("nan"), device="cuda")
    sc.paged_attention(q, k, v, table, _ints(past), cap=cap, out=got)
    ref.check_attention(got, (out, bound + 1.05 * 2 * E * float(vv.abs().max()), finite), f"{dtype} {L} {cap}")
