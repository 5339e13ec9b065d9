"""What 16-bit types lose in the weights, seen in fp32 outputs: nothing that their own rounding to 16 bits would hide.

Tolerance: tests/attention_ref.py's, with the weights' rounding as documented for few rows and for fp32 outputs: twice the bits, so 2^-16
of a weight in bf16 (half a unit, 2^-8, of what 2^-8 left) and 2^-22 in fp16, whose small weights the reference counts apart."""
import pytest
import torch

import attention_ref as ref
from test_gpu_attention import _check, _gen

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(autouse=True)
def twice_the_bits(monkeypatch):
    for t in TYPES:
        rel, tiny = ref.ROUND[t]
        monkeypatch.setitem(ref.ROUND, t, (rel * rel, tiny))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [32, 64, 80, 128, 192, 256])
def test_few_rows(dtype, D):
    g = _gen(D)
    _check(g, dtype, 2, 4, 2, D, 1, 32, [30, 500], out_f32=True)
    _check(g, dtype, 2, 4, 2, D, 5, 32, [0, 333], out_f32=True, spread=3.0)
    _check(g, dtype, 1, 4, 1, D, 4, 64, [700], out_f32=True, window=90, prefix=[20])
    _check(g, dtype, 1, 16, 1, D, 1, 64, [3000], out_f32=True, extra=9)  # in pieces
    if D <= 128:
        _check(g, dtype, 1, 4, 1, D, 8, 16, [100], out_f32=True, cap=20.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [32, 64, 80, 128, 192, 256])
def test_many_rows(dtype, D):
    g = _gen(D)
    _check(g, dtype, 1, 4, 1, D, 70, 16, [200], out_f32=True)
    _check(g, dtype, 2, 4, 2, D, 150, 64, [0, 90], out_f32=True, lengths=[150, 77], spread=3.0)
    _check(g, dtype, 1, 2, 1, D, 130, 64, [1000], extra=30, out_f32=True, window=300, prefix=[40])  # in pieces
    _check(g, dtype, 2, 2, 2, D, 140, 256, [0, 60], lengths=[140, 129], window=50, prefix=[5, 0], cap=8.0, out_f32=True, strided=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_infinities_in_part_of_the_rows(dtype, D):
    """The second walk, with both operands."""
    g = _gen(D + 1)

    def change(q, k, v, table):
        v[int(table[0, 1]), 0, 3, 5] = float("inf")
        v[int(table[0, 1]), 1, 7, 4] = float("nan")

    _check(g, dtype, 1, 4, 2, D, 3, 16, [19], change=change, out_f32=True)
    _check(g, dtype, 1, 4, 2, D, 150, 16, [0], change=change, out_f32=True)
    _check(g, dtype, 1, 4, 2, D, 150, 64, [0], change=change, out_f32=True, window=10)
