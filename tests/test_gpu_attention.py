"""The attention operators on the GPU against their definitions in float64, every output within the error that their
arithmetic may make (tests/attention_ref.py): the sizes, masks, strides and pages where they can go wrong."""
import numpy as np
import pytest
import torch

import attention_ref as ref
import sparse_weight_direct_amd as sc

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAN = float("nan")
INF = float("inf")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _strided(t, pad=3):
    """The same values as a view with gaps between rows and batches, starting at an odd offset."""
    *outer, L = t.shape
    big = torch.full([*outer[:-1], outer[-1] + 2, L + pad], NAN, dtype=t.dtype, device=t.device)
    view = big[..., 1:-1, 1:L + 1]
    view.copy_(t)
    return view


def _cache(g, dtype, G, D, P, past, lengths, L, extra=0):
    """Pools full of NaN but for the positions that there are, and their table (pages in any order)."""
    B = len(past)
    ends = [max(0, p) + (L if lengths is None else min(max(n, 0), L)) for p, n in zip(past, lengths or [L] * B)]
    width = max(1, max(-(-e // P) for e in ends)) + extra
    pages = B * width + 2
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = order[:B * width].view(B, width).contiguous()
    k = torch.full((pages, G, P, D), NAN, dtype=dtype, device="cuda")
    v = torch.full((pages, G, D, P), NAN, dtype=dtype, device="cuda")
    for b, e in enumerate(ends):
        for t0 in range(0, e, P):
            n = min(P, e - t0)
            page = int(table[b, t0 // P])
            k[page, :, :n] = _randn(g, G, n, D, dtype=dtype)
            v[page, :, :, :n] = _randn(g, G, D, n, dtype=dtype)
    return k, v, table


def _check(g, dtype, B, H, G, D, L, P, past, lengths=None, strided=False, extra=0, out_f32=False, change=None, spread=1.0, **kw):
    k, v, table = _cache(g, dtype, G, D, P, past, lengths, L, extra)
    q = _randn(g, B, H * D, L, dtype=dtype, scale=spread)
    if change:
        change(q, k, v, table)
    slopes = _randn(g, H).abs() if kw.pop("slopes", False) else None
    prefix = kw.pop("prefix", None)
    want = ref.paged_attention(q, k, v, table, _ints(past), lengths, slopes=slopes, prefix=prefix,
                               out_dtype=torch.float32 if out_f32 else None, **kw)
    if lengths is not None:
        for b, n in enumerate(lengths):
            q[b, :, max(0, min(n, L)):] = NAN
    if strided:
        q = _strided(q)
    out = torch.full((B, H * D, L), NAN, dtype=torch.float32 if out_f32 else dtype, device="cuda")
    if strided:
        out = _strided(out)
    got = sc.paged_attention(q, k, v, table, _ints(past), lengths=None if lengths is None else _ints(lengths), slopes=slopes,
                             prefix=None if prefix is None else _ints(prefix), out=out, **kw)
    assert got is out
    ref.check_attention(out, want, f"{dtype} {B} {H} {G} {D} {L} {P} {past} {kw}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [8, 16, 40, 64, 72, 96, 128, 136, 192, 256])
def test_head_dims(dtype, D):
    g = _gen(D)
    _check(g, dtype, 2, 4, 2, D, 1, 16, [37, 0])
    _check(g, dtype, 2, 3, 1, D, 20, 32, [5, 90])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
def test_pages(dtype, P):
    g = _gen(P)
    _check(g, dtype, 3, 4, 2, 64, 1, P, [0, P - 1, 3 * P + 5])
    _check(g, dtype, 3, 4, 2, 64, 33, P, [0, P - 1, 3 * P + 5], extra=2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [1, 2, 3, 7, 15, 16, 17, 31, 33, 63, 64, 65, 127, 130, 200, 257])
def test_chunk_lengths(dtype, L):
    g = _gen(L)
    _check(g, dtype, 2, 6, 2, 64, L, 64, [0, 71])
    _check(g, dtype, 2, 2, 2, 40, L, 16, [0, 71], lengths=[L, L // 2])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,G", [(1, 1), (2, 1), (7, 1), (16, 1), (17, 1), (33, 1), (70, 1), (5, 5), (24, 8), (64, 4)])
def test_heads(dtype, H, G):
    g = _gen(H)
    _check(g, dtype, 2, H, G, 32, 1, 32, [100, 3])
    _check(g, dtype, 1, H, G, 32, 5, 32, [60])
    _check(g, dtype, 1, H, G, 32, 70, 32, [11])


@pytest.mark.parametrize("dtype", TYPES)
def test_unequal_lengths_idle_and_empty(dtype):
    g = _gen(1)
    _check(g, dtype, 7, 4, 2, 64, 40, 32, [0, 5, 100, -1, 33, 7, 64], lengths=[40, 0, 1, 40, -3, 99, 17])
    _check(g, dtype, 4, 4, 2, 64, 1, 32, [0, -1, 10 ** 6, 64])
    _check(g, dtype, 3, 4, 2, 64, 150, 64, [0, 300, -5], lengths=[1, 150, 150])
    k, v, table = _cache(g, dtype, 2, 64, 32, [4], None, 1)
    assert sc.paged_attention_step(torch.empty(0, 256, dtype=dtype, device="cuda"), k, v, table[:0], _ints([])).shape == (0, 256)
    assert sc.paged_attention(torch.empty(1, 256, 0, dtype=dtype, device="cuda"), k, v, table, _ints([4])).shape == (1, 256, 0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("window", [1, 2, 16, 31, 32, 33, 64, 100, 1000, 2 ** 40])
def test_window(dtype, window):
    g = _gen(window % 1000)
    kw = dict(window=window)
    _check(g, dtype, 2, 4, 2, 64, 1, 16, [0, 300], **kw)
    _check(g, dtype, 2, 4, 2, 64, 9, 16, [50, 300], **kw)
    _check(g, dtype, 2, 4, 2, 64, 140, 64, [0, 300], **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("prefix", [[0, -4], [1, 5], [33, 64], [200, 10 ** 6]])
@pytest.mark.parametrize("window", [0, 20])
def test_prefix(dtype, prefix, window):
    g = _gen(prefix[0])
    _check(g, dtype, 2, 4, 2, 64, 1, 16, [130, 300], prefix=prefix, window=window)
    _check(g, dtype, 2, 4, 2, 64, 100, 32, [0, 300], prefix=prefix, window=window)
    _check(g, dtype, 2, 4, 2, 64, 170, 32, [0, 300], prefix=prefix, window=window, lengths=[77, 170])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [1, 6, 40, 150])
def test_cap_bias_scale(dtype, L):
    g = _gen(L)
    _check(g, dtype, 2, 6, 2, 64, L, 32, [17, 200], cap=5.0, spread=4.0)
    _check(g, dtype, 2, 6, 2, 64, L, 32, [17, 200], slopes=True)
    _check(g, dtype, 2, 6, 2, 64, L, 32, [17, 200], slopes=True, cap=50.0, window=60, prefix=[3, 90], scale=-0.3)
    _check(g, dtype, 2, 6, 2, 64, L, 32, [17, 200], scale=0.0)
    _check(g, dtype, 2, 6, 2, 64, L, 32, [17, 200], spread=12.0)  # few weights count


@pytest.mark.parametrize("dtype", TYPES)
def test_long_contexts_in_pieces(dtype):
    """A context that several workgroups share (and wavefronts that find none of it)."""
    g = _gen(5)
    for past in ([3000], [0], [130], [1500, 2]):
        _check(g, dtype, len(past), 4, 2, 64, 1, 64, past, extra=40)
        _check(g, dtype, len(past), 4, 2, 128, 3, 16, past, extra=40)
        _check(g, dtype, len(past), 4, 1, 64, 50, 64, past, extra=9)
    _check(g, dtype, 1, 2, 1, 256, 1, 64, [2000], window=700, prefix=[70], extra=5)
    _check(g, dtype, 2, 2, 1, 64, 1, 64, [2000, -1], extra=5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [1, 4, 60, 140])
def test_missing_pages(dtype, L):
    """Entries of the table outside the pool hide their positions; a row may be left with nothing."""
    g = _gen(L)

    def change(q, k, v, table):
        table[0, 1] = -1
        table[1, 0] = k.shape[0]
        table[2, :] = -7
        table[3, 2:] = 2 ** 31 - 1

    _check(g, dtype, 4, 4, 2, 64, L, 16, [40, 70, 33, 90], change=change)
    _check(g, dtype, 4, 4, 2, 64, L, 64, [200, 270, 133, 300], change=change, window=50)


@pytest.mark.parametrize("dtype", TYPES)
def test_past_the_table(dtype):
    """Positions past the table's end are not there."""
    g = _gen(9)
    k, v, table = _cache(g, dtype, 2, 64, 16, [48], None, 16)
    q = _randn(g, 1, 256, 40, dtype=dtype)
    want = ref.paged_attention(q, k, v, table, _ints([48]))
    ref.check_attention(sc.paged_attention(q, k, v, table, _ints([48])), want)
    want = ref.paged_attention(q, k, v, table, _ints([64]))
    ref.check_attention(sc.paged_attention(q, k, v, table, _ints([64])), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_infinities_that_nobody_sees(dtype, value, D):
    """An infinite key or value spoils the rows that see it, and no other."""
    g = _gen(D)

    def change(q, k, v, table):
        v[int(table[0, 1]), 0, 3, 5] = value  # position P + 5: the rows from there on see it
        v[int(table[0, 1]), 1, 7, 4] = value

    _check(g, dtype, 1, 4, 2, D, 40, 16, [0], change=change)
    _check(g, dtype, 1, 4, 2, D, 3, 16, [19], change=change)
    _check(g, dtype, 1, 4, 2, D, 40, 16, [0], change=change, window=4)
    _check(g, dtype, 1, 4, 2, D, 150, 64, [0], change=change, window=10)
    _check(g, dtype, 1, 2, 2, D, 150, 64, [40], change=change, window=10, prefix=[30])

    def keys(q, k, v, table):
        k[int(table[0, 2]), 0, 4, 3] = NAN  # past what the rows see

    _check(g, dtype, 1, 4, 2, D, 36, 16, [0], lengths=[36], change=keys, window=0, extra=0) if value != value else None
    for n in (3, 130):  # NaN past the end, in the last page: _cache leaves it there
        _check(g, dtype, 2, 4, 2, D, n, 64, [13, 20])


@pytest.mark.parametrize("dtype", TYPES)
def test_extreme_scores(dtype):
    """Scores far from 0, and an infinite one in a visible place."""
    g = _gen(3)

    def change(q, k, v, table):
        q[:, :, 0] = 30.0

    _check(g, torch.float32, 1, 2, 1, 64, 3, 16, [20], change=change, spread=5.0)
    k, v, table = _cache(g, dtype, 1, 64, 16, [20], None, 1)
    q = torch.zeros(1, 64, dtype=dtype, device="cuda")
    q[0, 0] = 1.0
    page = int(table[0, 0])
    k[page, 0, 3] = 0
    k[page, 0, 3, 0] = -INF  # a weight of 0
    got = sc.paged_attention_step(q, k, v, table, _ints([20]))
    k[page, 0, 3, 0] = -200.0 if dtype != torch.float32 else -1e4  # the same: exp of it is 0 beside the others
    same = ref.paged_attention(q[:, :, None], k, v, table, _ints([20]), scale=100.0)
    ref.check_attention(sc.paged_attention_step(q, k, v, table, _ints([20]), scale=100.0)[:, :, None], same)
    assert torch.isfinite(got).all()
    k[page, 0, 3, 0] = INF
    assert torch.isnan(sc.paged_attention_step(q, k, v, table, _ints([20]))).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_strides_and_views(dtype):
    g = _gen(4)
    for L in (2, 20, 150):
        _check(g, dtype, 2, 4, 2, 64, L, 32, [30, 3], strided=True)
    # parts of one projection, channels of single positions apart, pages of keys and values side by side, a wider table's rows
    k, v, table = _cache(g, dtype, 2, 64, 32, [70, 9], None, 1)
    both = torch.empty(k.shape[0], 2, k[0].numel(), dtype=dtype, device="cuda")
    both[:, 0], both[:, 1] = k.flatten(1), v.flatten(1)
    kv, vv = both[:, 0].view(k.shape[0], 2, 32, 64), both[:, 1].view(k.shape[0], 2, 64, 32)
    wide = torch.full((2, table.shape[1] + 3), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    q = _randn(g, 2, 256, dtype=dtype)
    want = ref.paged_attention(q[:, :, None], k, v, table, _ints([70, 9]))
    spaced = torch.full((2, 256, 3), NAN, dtype=dtype, device="cuda")
    spaced[:, :, 1] = q
    out = torch.full((2, 256, 5), NAN, dtype=dtype, device="cuda")
    sc.paged_attention_step(spaced[:, :, 1], kv, vv, wide[:, :table.shape[1]], _ints([70, 9]), out=out[:, :, 2])
    ref.check_attention(out[:, :, 2:3], want)
    assert torch.isnan(out[:, :, [0, 1, 3, 4]]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_float32_output_of_16_bit_queries(dtype):
    g = _gen(8)
    _check(g, dtype, 2, 4, 2, 64, 1, 32, [30, 500], out_f32=True)
    _check(g, dtype, 2, 4, 2, 64, 1, 32, [30, 5000], out_f32=True)
    _check(g, dtype, 2, 4, 2, 64, 170, 32, [30, 3], out_f32=True)


def test_same_inputs_give_the_same_bits():
    g = _gen(11)
    for L, past in ((1, 5000), (40, 700), (300, 100)):
        k, v, table = _cache(g, torch.bfloat16, 2, 128, 64, [past], None, L)
        q = _randn(g, 1, 8 * 128, L, dtype=torch.bfloat16)
        a = sc.paged_attention(q, k, v, table, _ints([past]))
        for _ in range(3):
            assert torch.equal(a, sc.paged_attention(q, k, v, table, _ints([past])))


# ---- append


def _check_append(g, dtype, cache, B, H, G, D, L, P, past, lengths=None, pairs=None, axes=1, interleaved=False, strided=False,
                  in_place=False, missing=False, far=100_000, no_q=False):
    width = max(1, max(-(-(max(0, p) + L) // P) for p in past))
    pages = B * width + 2
    table = torch.randperm(pages, generator=g, device="cuda")[:B * width].to(torch.int32).view(B, width).contiguous()
    if missing:
        table[0, 0], table[-1, -1] = -1, pages
    k_pages, v_pages = _randn(g, pages, G, P, D, dtype=cache), _randn(g, pages, G, D, P, dtype=cache)
    q, k, v = (_randn(g, B, n * D, L, dtype=dtype) for n in (H, G, G))
    pairs = D // 2 if pairs is None else pairs
    freqs = torch.pow(10000.0, -torch.arange(pairs, device="cuda", dtype=torch.float64) / max(pairs, 1)) if pairs else None
    ax = (torch.arange(pairs, device="cuda") % (axes + 1) - int(pairs > 4)).to(torch.int32) if axes > 1 else None  # -1: it stays
    positions = torch.randint(-far, far, (B, axes, L), generator=g, device="cuda", dtype=torch.int32) if axes > 1 else None
    want = ref.cache_append(k, v, k_pages, v_pages, table, _ints(past), None if no_q else q, freqs, ax, positions, interleaved, lengths)
    if lengths is not None:
        for b, n in enumerate(lengths):
            for t in (q, k, v):
                t[b, :, max(0, min(n, L)):] = NAN
    if strided:
        q, k, v = _strided(q), _strided(k), _strided(v)
    out = None
    if not no_q:
        out = q if in_place else torch.full((B, H * D, L), NAN, dtype=cache, device="cuda")
        if strided and not in_place:
            out = _strided(out)
    got = sc.cache_append(k, v, k_pages, v_pages, table, _ints(past), q=None if no_q else q, freqs=freqs, axes=ax, positions=positions,
                          interleaved=interleaved, lengths=None if lengths is None else _ints(lengths), out=out)
    assert got is out
    if not no_q:
        ref.assert_near(got, want[0], want[1], "q")
    ref.assert_near(k_pages, want[2], want[3], "k")
    assert torch.equal(ref.wide(v_pages), want[4])


CACHES = [(torch.float32, torch.float32), (torch.float32, torch.bfloat16), (torch.float32, torch.float16),
          (torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16)]


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("L", [1, 2, 7, 8, 15, 16, 17, 63, 64, 65, 130, 200])
def test_append_lengths(dtype, cache, L):
    g = _gen(L)
    _check_append(g, dtype, cache, 2, 4, 2, 64, L, 32, [0, 45])
    _check_append(g, dtype, cache, 3, 2, 1, 40, L, 16, [3, 64, 129], lengths=[L, 0, (L + 1) // 2], missing=True)


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("D", [8, 24, 64, 128, 136, 256])
def test_append_dims_and_pairs(dtype, cache, D):
    g = _gen(D)
    for L in (1, 20, 70):
        for pairs in sorted({0, 1, D // 4, D // 2}):
            _check_append(g, dtype, cache, 2, 3, 3, D, L, 64, [5, 60], pairs=pairs, interleaved=bool(pairs % 2))


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_axes(dtype, cache, axes, interleaved):
    g = _gen(axes)
    for L in (1, 9, 40, 90):
        _check_append(g, dtype, cache, 2, 9, 2, 64, L, 64, [0, 33], axes=axes, interleaved=interleaved)
    _check_append(g, dtype, cache, 1, 2, 2, 64, 40, 64, [0], axes=axes, interleaved=interleaved, far=2 ** 30)


@pytest.mark.parametrize("dtype,cache", CACHES)
@pytest.mark.parametrize("P", [16, 32, 64, 128, 256])
def test_append_pages_idle_and_strides(dtype, cache, P):
    g = _gen(P)
    for L in (1, 5, 40, 100):
        _check_append(g, dtype, cache, 4, 4, 2, 32, L, P, [0, P - 1, -2, 2 * P + 7], lengths=None if L == 1 else [L, L - 1, 3, 1], strided=L > 1)
        if dtype == cache:
            _check_append(g, dtype, cache, 2, 4, 2, 32, L, P, [9, 3 * P], in_place=True)
        _check_append(g, dtype, cache, 2, 4, 2, 32, L, P, [9, 3 * P], no_q=True)


def test_append_past_the_table():
    g = _gen(2)
    for L in (4, 100):
        k_pages, v_pages = _randn(g, 3, 1, 16, 32), _randn(g, 3, 1, 32, 16)
        table = _ints([[1], [2], [0]])
        k, v, q = (_randn(g, 3, 32, L) for _ in range(3))
        past = _ints([14, 16, 17])  # partly past it, wholly past it, idle
        freqs = torch.ones(4, dtype=torch.float64, device="cuda")
        want = ref.cache_append(k, v, k_pages, v_pages, table, past, q, freqs)
        got = sc.cache_append(k, v, k_pages, v_pages, table, past, q=q, freqs=freqs)
        ref.assert_near(got, want[0], want[1])
        ref.assert_near(k_pages, want[2], want[3])
        assert torch.equal(ref.wide(v_pages), want[4])
        assert (got[2] == 0).all()


def test_append_step_with_any_strides():
    g = _gen(6)
    qkv = _randn(g, 5, 8 * 32, 3, dtype=torch.bfloat16)[:, :, 1]
    q, k, v = qkv[:, :128], qkv[:, 128:192], qkv[:, 192:]
    k_pages, v_pages = _randn(g, 9, 2, 16, 32, dtype=torch.bfloat16), _randn(g, 9, 2, 32, 16, dtype=torch.bfloat16)
    table = torch.randperm(9, generator=g, device="cuda")[:5].to(torch.int32).view(5, 1)
    past = _ints([0, 3, 15, 7, -1])
    freqs = torch.pow(100.0, -torch.arange(16, device="cuda", dtype=torch.float64) / 16)
    want = ref.cache_append(k[:, :, None], v[:, :, None], k_pages, v_pages, table, past, q[:, :, None], freqs)
    got = sc.cache_append_step(k, v, k_pages, v_pages, table, past, q=q, freqs=freqs)
    ref.assert_near(got[:, :, None], want[0], want[1])
    ref.assert_near(k_pages, want[2], want[3])
    assert torch.equal(ref.wide(v_pages), want[4])


# ---- copies


@pytest.mark.parametrize("dtype", TYPES + [torch.uint8, torch.float64])
@pytest.mark.parametrize("shape", [(1, 5, 3), (2, 9, 16), (3, 40, 2, 16, 24), (24, 30, 4096), (2, 7, 8195), (1, 4, 70000)])
def test_copy(dtype, shape):
    g = _gen(shape[1])
    pool = torch.randint(0, 200, shape, generator=g, device="cuda").to(dtype)
    order = torch.randperm(shape[1], generator=g, device="cuda").to(torch.int32)
    n = shape[1] // 2
    source, target = order[:n].clone(), order[n:2 * n].clone()
    want = pool.clone()
    want[:, target.long()] = pool[:, source.long()]
    got = sc.cache_copy(pool, source, target)
    assert got is pool and torch.equal(pool, want)


def test_copy_leaves_out_bad_pairs_and_takes_views():
    g = _gen(0)
    big = _randn(g, 4, 6, 50, dtype=torch.bfloat16)
    pool = big[1:3, ::2, 1:33]  # pages of 64 bytes, 200 apart, at an odd offset
    want = big.clone()
    want[1:3, 2, 1:33] = big[1:3, 4, 1:33]
    sc.cache_copy(pool, _ints([2, -1, 0, 3, 1, 2 ** 31 - 1]), _ints([1, 0, 7, 0, -5, 0]))
    assert torch.equal(big, want)
    for empty in (_ints([]),):
        sc.cache_copy(pool, empty, empty)
    sc.cache_copy(big[:0], _ints([0]), _ints([1]))
    sc.cache_copy(big, _ints([1]), _ints([1]))  # onto itself: nothing
    assert torch.equal(big, want)


# ---- norms


def _check_norm(g, dtype, B, C, L, post=True, pre=True, gate=None, center=False, strided=False, in_place=False, y=True, scale=0.7,
                eps=1e-6, size=1.0, affine=True):
    x = _randn(g, B, C, L, dtype=dtype, scale=2.0 * size)
    yv = _randn(g, B, C, L, dtype=dtype, scale=size) if y else None
    w, b, pw, pb = (_randn(g, C) if affine or i == 2 else None for i in range(4))
    w, b = (w, b) if pre else (None, None)
    pw, pb = (pw, pb) if post and y else (None, None)
    gt = None if gate is None else _randn(g, B, C, *((L,) if gate == "all" else ()), dtype=dtype)
    kw = dict(weight=w, bias=b, post_weight=pw, post_bias=pb, scale=scale, eps=eps, center=center)
    want = ref.residual_norm(x, yv, gate=gt, normed=pre, **kw)
    if strided:
        x, yv, gt = _strided(x), None if yv is None else _strided(yv), gt if gt is None or gt.dim() == 2 else _strided(gt)
    x0 = x
    sum_ = x if in_place else torch.full((B, C, L), NAN, dtype=dtype, device="cuda") if y else None
    out = None
    if pre:
        out = yv if in_place and y else torch.full((B, C, L), NAN, dtype=dtype, device="cuda")
    if strided and not in_place:
        sum_, out = None if sum_ is None else _strided(sum_), None if out is None else _strided(out)
    r, h = sc.residual_norm(x, yv, gate=gt, sum=sum_ if y else None, out=out, **kw)
    assert r is (sum_ if y else x0) and h is out
    ref.assert_near(r, want[0], want[1], "sum")
    if pre:
        ref.assert_near(h, want[2], want[3], "out")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("C", [1, 2, 7, 64, 100, 511, 768, 1025, 2048, 4097, 8200])
def test_norm_channels(dtype, C):
    g = _gen(C)
    for L in (1, 5, 33):
        _check_norm(g, dtype, 2, C, L)
        _check_norm(g, dtype, 2, C, L, center=True, gate="channels")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [1, 2, 3, 4, 7, 8, 9, 15, 16, 17, 31, 32, 33, 64, 100, 257])
def test_norm_lengths(dtype, L):
    g = _gen(L)
    _check_norm(g, dtype, 3, 96, L, gate="all")
    _check_norm(g, dtype, 3, 96, L, post=False)
    _check_norm(g, dtype, 3, 96, L, pre=False, gate="channels")
    _check_norm(g, dtype, 3, 96, L, y=False)
    _check_norm(g, dtype, 3, 96, L, y=False, center=True, affine=False)
    _check_norm(g, dtype, 3, 96, L, strided=True, gate="all", center=True)
    _check_norm(g, dtype, 3, 96, L, in_place=True)
    _check_norm(g, dtype, 3, 2000, L, in_place=True, center=True)


@pytest.mark.parametrize("dtype", TYPES)
def test_norm_values(dtype):
    g = _gen(1)
    for size in (1e-3, 1.0, 100.0):
        _check_norm(g, dtype, 2, 300, 20, size=size)
        _check_norm(g, dtype, 2, 300, 20, size=size, eps=0.1, center=True)
    z = torch.zeros(2, 64, 8, dtype=dtype, device="cuda")
    r, h = sc.residual_norm(z, z, weight=torch.ones(64, device="cuda"), post_weight=torch.ones(64, device="cuda"))
    assert (r == 0).all() and (h == 0).all()
    # what is not finite stays in its own position
    x = _randn(g, 2, 64, 20, dtype=dtype)
    x[0, 3, 4], x[1, 60, 19] = INF, NAN
    want = ref.residual_norm(torch.where(torch.isfinite(x), x, 0.0), weight=torch.ones(64))
    _, h = sc.residual_norm(x, weight=torch.ones(64, device="cuda"))
    keep = torch.ones(2, 64, 20, dtype=torch.bool)
    keep[0, :, 4], keep[1, :, 19] = False, False
    h = ref.wide(h)
    assert torch.isfinite(h[keep]).all() and ((h - want[2]).abs() <= want[3])[keep].all()
    assert not torch.isfinite(h[0, 3, 4]) and not torch.isfinite(h[1, :, 19]).any()


@pytest.mark.parametrize("dtype", TYPES)
def test_norm_step_with_any_strides(dtype):
    g = _gen(3)
    for C in (96, 2048, 4100):
        x, y = _randn(g, 5, C, 2, dtype=dtype), _randn(g, 5, C, 2, dtype=dtype)
        w = _randn(g, C)
        want = ref.residual_norm(x, y, weight=w, post_weight=w)
        for i in range(2):
            r, h = sc.residual_norm_step(x[:, :, i], y[:, :, i], weight=w, post_weight=w)
            ref.assert_near(r, want[0][:, :, i], want[1][:, :, i])
            ref.assert_near(h, want[2][:, :, i], want[3][:, :, i])
            r, h = sc.residual_norm_step(x[:, :, i].contiguous(), y[:, :, i].contiguous(), weight=w, post_weight=w)
            ref.assert_near(r, want[0][:, :, i], want[1][:, :, i])
            ref.assert_near(h, want[2][:, :, i], want[3][:, :, i])


def test_norm_empty():
    x = torch.empty(0, 64, 8, device="cuda")
    r, h = sc.residual_norm(x, x, weight=torch.ones(64, device="cuda"))
    assert r.shape == x.shape and h.shape == x.shape
    x = torch.empty(2, 64, 0, device="cuda")
    assert sc.residual_norm(x, weight=torch.ones(64, device="cuda"))[1].shape == x.shape
