"""The forms of the sequence operators' kernels that only large calls take: the scan without reading ahead (one walk, and
segments) and the adapters' second product with four tiles of positions side by side.  tests/test_sequence_plan.py
holds that these sizes take them."""
import pytest
import torch

import sequence_ref as ref
import sparse_weight_direct_amd as sc
from test_gpu_sequence import TYPES, _check_scan, _gen, _ints, _randn, _strided

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,strided", [(20, False), (16, True)])
def test_scan_without_reading_ahead(dtype, N, strided):
    _check_scan(_gen(N), dtype, 9, 1023, 520, N, 1, lengths=[520, 0, 1, 257, 300, 256, 519, 400, 33], state="inplace", strided=strided)


@pytest.mark.parametrize("dtype", TYPES)
def test_scan_in_segments_without_reading_ahead(dtype):
    _check_scan(_gen(21), dtype, 2, 512, 2311, 20, 1, lengths=[2311, 1500], slots=[2, 0], pool=3, state="inplace")
    _check_scan(_gen(22), dtype, 1, 1024, 2500, 16, 4, state="both", strided=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R", [4, 16])
def test_adapter_tiles_side_by_side(dtype, R):
    """The last set of four tiles has one, the last tile is not whole, and a tile's values are up to 2^20 times the
    next one's (fp16 holds the intermediate with an exponent a position)."""
    g = _gen(R)
    tile = 64 if dtype == torch.float32 else 128
    B, C, M, L, n = 64, 12, 150, 21 * tile - 37, 3
    x = _randn(g, B, C, L) * torch.exp2(torch.arange(L, device="cuda") // tile % 5 * 5.0 - 14.0)
    x, base = x.to(dtype), _randn(g, B, M, L, dtype=dtype)
    down, up = _randn(g, n, R, C, dtype=dtype, scale=C ** -0.5), _randn(g, n, M, R, dtype=dtype, scale=R ** -0.5)
    scale = _randn(g, n)
    index = [(k * 7) % 5 - 1 for k in range(B)]  # -1 and 3: none
    want, bound = ref.adapter(x, down, up, index, scale, base)
    if R == 4:
        x, out = _strided(x), _strided(base)
        sc.adapter_apply(x, down, up, _ints(index), scale=scale, base=out, out=out)
    else:
        out = sc.adapter_apply(x, down, up, _ints(index), scale=scale, base=base)
    ref.assert_within(out, want, bound, "adapter")


def _adapter_within(x, down, up, index, scale, base, out):
    """tests/sequence_ref.py's adapter and its bound, in float64 on the GPU for the sizes that take long on a CPU."""
    low = 2.0 ** -16 if x.dtype != torch.float32 else 0.0
    rel, tiny = ref.ROUND[x.dtype]
    C, R = x.shape[1], down.shape[1]
    for b, r in enumerate(index):
        X, v, err = x[b].double(), base[b].double(), torch.zeros((), dtype=torch.float64, device="cuda")
        if 0 <= r < down.shape[0]:
            s, d, u = float(scale[r]), down[r].double(), up[r].double()
            v = v + s * (u @ (d @ X))
            err = ((C + R + 8) * ref.U + low) * abs(s) * (u.abs() @ (d.abs() @ X.abs())) + 2 * ref.U * v.abs()
        assert ((out[b].double() - v).abs() <= err + rel * (v.abs() + err) + tiny).all(), b


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,M,C,R,wide", [(8, 3000, 1030, 16, True), (16, 1500, 600, 7, True), (24, 130, 600, 20, False)])
def test_adapter_pieces_of_the_channels(dtype, B, M, C, R, wide):
    """The first product cut into 4 and 2 pieces of C, whose sums the second adds, with and without four tiles side by side."""
    g = _gen(B)
    tile = 64 if dtype == torch.float32 else 128
    L, n = (16 if wide else 6) * tile - 5, 3
    x, base = _randn(g, B, C, L, dtype=dtype), _randn(g, B, M, L, dtype=dtype)
    down, up = _randn(g, n, R, C, dtype=dtype, scale=C ** -0.5), _randn(g, n, M, R, dtype=dtype, scale=R ** -0.5)
    scale, index = _randn(g, n), [k % 5 - 1 for k in range(B)]
    out = sc.adapter_apply(x, down, up, _ints(index), scale=scale, base=base)
    _adapter_within(x, down, up, index, scale, base, out)
    sc.adapter_apply(x, down, up, _ints(index), scale=scale, base=base, out=base)
    assert torch.equal(out, base)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,M,C,tiles", [(64, 150, 12, 21), (8, 3000, 1030, 16), (16, 1500, 600, 16)])
def test_adapter_infinite_weights_with_tiles_side_by_side(dtype, B, M, C, tiles):
    """R values of one sign: an infinite weight makes its row infinite at every position, and the others stay as they are."""
    g = _gen(B + 1)
    L, R = tiles * (64 if dtype == torch.float32 else 128) - 37, 9
    x = (torch.rand(B, C, L, generator=g, device="cuda") + 0.5).to(dtype)
    down = ((torch.rand(2, R, C, generator=g, device="cuda") + 0.5) / C).to(dtype)
    up, base, index = _randn(g, 2, M, R, dtype=dtype), _randn(g, B, M, L, dtype=dtype), [k % 3 - 1 for k in range(B)]
    clean = sc.adapter_apply(x, down, up, _ints(index), base=base)
    up[1, 5, 0], up[1, M - 1, R - 1] = float("inf"), -float("inf")
    out = sc.adapter_apply(x, down, up, _ints(index), base=base)
    one = torch.tensor(index, device="cuda") == 1
    assert (out[one, 5] == float("inf")).all() and (out[one, M - 1] == -float("inf")).all()
    out[one, 5], out[one, M - 1] = clean[one, 5], clean[one, M - 1]
    assert torch.equal(out, clean)
