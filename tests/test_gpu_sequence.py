"""The sequence operators on the GPU against their definitions in float64, every output within the
error that their arithmetic may make (tests/sequence_ref.py): the sizes, masks, strides and states
where they can go wrong."""
import numpy as np
import pytest
import torch

import sequence_ref as ref
import sparse_weight_direct_amd as sc

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAN = float("nan")


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _strided(t, pad=3):
    """The same values as a view with gaps between rows and batches, starting at an odd offset."""
    *outer, L = t.shape
    big = torch.full([*outer[:-1], outer[-1] + 2, L + pad], NAN, dtype=t.dtype, device=t.device)
    view = big[..., 1:-1, 1:L + 1]
    view.copy_(t)
    return view


def _past(t, lengths, value):
    """`value` in every position past its sequence's length."""
    t = t.clone()
    for b, n in enumerate(lengths):
        t[b, ..., max(0, min(int(n), t.shape[-1])):] = value
    return t


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---- the causal convolution


def _check_conv(g, dtype, B, D, L, K, silu=True, bias=True, lengths=None, slots=None, pool=None, state="none",
                strided=False):
    x = _randn(g, B, D, L, dtype=dtype)
    w = _randn(g, D, K, scale=K ** -0.5)
    bv = _randn(g, D) if bias else None
    n = pool or B
    first = _randn(g, n, D, K - 1, dtype=dtype) if state != "none" else None
    last = first.clone() if state == "inplace" else _randn(g, n, D, K - 1, dtype=dtype) if state == "both" else None
    want, bound, P = ref.causal_conv(x, w, bv, silu, lengths, slots, first, last)
    given = first if state != "inplace" else last
    if lengths is not None:
        x = _past(x, lengths, NAN)
    if strided:
        x = _strided(x)
    out = torch.full((B, D, L), NAN, dtype=dtype, device="cuda")
    if strided:
        out = _strided(out)
    got = sc.causal_conv(x, w, bv, silu=silu, lengths=None if lengths is None else _ints(lengths),
                         slots=None if slots is None else _ints(slots), initial_state=given, final_state=last, out=out)
    assert got is out
    ref.assert_within(out, want, bound, "conv")
    if last is not None:
        np.testing.assert_array_equal(ref.f64(last), P)  # inputs as they were


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 6, 7, 8])
def test_conv_taps_and_lengths(dtype, K):
    g = _gen(K)
    for L in (0, 1, 2, 7, 8, 9, 17, 64, 257, 1030):
        _check_conv(g, dtype, 2, 5, L, K, state="both")
    _check_conv(g, dtype, 2, 5, 33, K, silu=False, bias=False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [1700, 2041, 2048, 2049, 4090])
def test_conv_long_rows(dtype, L):
    _check_conv(_gen(L), dtype, 2, 3, L, 4, state="both")
    _check_conv(_gen(L), dtype, 3, 3, L, 3, lengths=[L, L - 5, 1], state="inplace", strided=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("strided", [False, True])
def test_conv_ragged_slots_and_states(dtype, strided):
    g = _gen(3)
    _check_conv(g, dtype, 7, 9, 41, 4, lengths=[41, 0, 1, 2, 3, 17, 100], state="inplace", strided=strided)
    _check_conv(g, dtype, 5, 9, 19, 4, lengths=[-5, 19, 1, 2, 8], slots=[7, -1, 2, 8, 0], pool=8, state="inplace",
                strided=strided)
    _check_conv(g, dtype, 5, 9, 23, 3, slots=[7, -1, 2, 8, 0], pool=8, state="both", strided=strided)
    _check_conv(g, dtype, 3, 64, 300, 4, state="both", strided=strided)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,D,K,pool,slots", [(1, 1, 4, None, None), (3, 37, 4, None, None), (2, 64, 2, None, None),
                                              (4, 130, 3, 6, [5, 0, 3, 1]), (4, 129, 8, 5, [4, -1, 99, 0]),
                                              (2, 16, 1, None, None), (5, 512, 4, None, None)])
def test_conv_step(dtype, B, D, K, pool, slots):
    g = _gen(B + D)
    wide = _randn(g, B, 2 * D, dtype=dtype)
    x = wide[:, D:]
    w, bv = _randn(g, D, K), _randn(g, D)
    state = _randn(g, pool or B, D, K - 1, dtype=dtype)
    want, bound, P = ref.causal_conv(x[:, :, None], w, bv, True, None, slots, state, state)
    out = sc.causal_conv_step(x, state, w, bv, slots=None if slots is None else _ints(slots))
    ref.assert_within(out[:, :, None], want, bound, "conv step")
    np.testing.assert_array_equal(ref.f64(state), P)


def test_conv_steps_repeat_the_prompt():
    g = _gen(9)
    B, D, L, K = 2, 70, 13, 4
    x, w, bv = _randn(g, B, D, L), _randn(g, D, K), _randn(g, D)
    whole = sc.causal_conv(x, w, bv)
    state = torch.zeros(B, D, K - 1, device="cuda")
    steps = torch.stack([sc.causal_conv_step(x[:, :, t], state, w, bv) for t in range(L)], 2)
    assert torch.equal(whole, steps)
    # and a prompt in two chunks, the state carried between them
    state.zero_()
    a = sc.causal_conv(x[:, :, :5], w, bv, initial_state=state, final_state=state)
    b = sc.causal_conv(x[:, :, 5:], w, bv, initial_state=state, final_state=state)
    assert torch.equal(whole, torch.cat([a, b], 2))


# ---- the scan


def _scan_inputs(g, dtype, B, D, L, N, G, z=True, skip=True, bias=True, softplus=True):
    s = {"x": _randn(g, B, D, L, dtype=dtype), "dt": _randn(g, B, D, L, dtype=dtype, scale=0.5),
         "A": -torch.exp(_randn(g, D, N, scale=0.7)), "B": _randn(g, B, G, N, L, dtype=dtype),
         "C": _randn(g, B, G, N, L, dtype=dtype), "D": _randn(g, D) if skip else None,
         "z": _randn(g, B, D, L, dtype=dtype) if z else None, "dt_bias": _randn(g, D) - 2 if bias else None}
    if not softplus:
        s["dt"], s["dt_bias"] = s["dt"].abs() * 0.3, s["dt_bias"].abs() * 0.1 if bias else None
    return s


def _check_scan(g, dtype, B, D, L, N, G=1, lengths=None, slots=None, pool=None, state="none", strided=False,
                softplus=True, **kw):
    s = _scan_inputs(g, dtype, B, D, L, N, G, softplus=softplus, **kw)
    n = pool or B
    first = _randn(g, n, D, N) if state != "none" else None
    last = first.clone() if state == "inplace" else _randn(g, n, D, N) if state == "both" else None
    want, bound, P, PB = ref.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"],
                                            softplus, lengths, slots, first, last)
    for k in ("x", "dt", "z", "B", "C"):
        if s[k] is not None:
            if lengths is not None:
                s[k] = _past(s[k], lengths, NAN)
            if strided:
                s[k] = _strided(s[k])
    out = torch.full((B, D, L), NAN, dtype=dtype, device="cuda")
    if strided:
        out = _strided(out)
    given = first if state != "inplace" else last
    sc.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                      softplus=softplus, lengths=None if lengths is None else _ints(lengths),
                      slots=None if slots is None else _ints(slots), initial_state=given, final_state=last, out=out)
    ref.assert_within(out, want, bound, "scan")
    if last is not None:
        ref.assert_within(last, P, PB, "scan state")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 511, 1025])
def test_scan_lengths(dtype, L):
    _check_scan(_gen(L), dtype, 2, 5, L, 16, state="both")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,G,D", [(1, 1, 3), (2, 1, 17), (5, 2, 34), (15, 1, 16), (16, 4, 64), (17, 1, 5), (24, 2, 32),
                                   (32, 1, 20), (64, 3, 51), (100, 1, 8), (256, 2, 6)])
def test_scan_states_and_groups(dtype, N, G, D):
    _check_scan(_gen(N), dtype, 2, D, 77, N, G, state="both")
    _check_scan(_gen(N), dtype, 1, D, 290, N, G)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("strided", [False, True])
def test_scan_ragged_slots_and_states(dtype, strided):
    g = _gen(4)
    _check_scan(g, dtype, 7, 18, 301, 16, 2, lengths=[301, 0, 1, 2, 16, 257, 999], state="inplace", strided=strided)
    _check_scan(g, dtype, 5, 18, 40, 12, 1, lengths=[-5, 40, 1, 33, 8], slots=[7, -1, 2, 8, 0], pool=8, state="inplace",
                strided=strided)
    _check_scan(g, dtype, 5, 9, 70, 16, 3, slots=[7, -1, 2, 8, 0], pool=8, state="both", strided=strided)


@pytest.mark.parametrize("kw", [dict(z=False), dict(skip=False), dict(bias=False), dict(softplus=False),
                                dict(z=False, skip=False, bias=False, softplus=False)])
def test_scan_without_its_options(kw):
    _check_scan(_gen(5), torch.float32, 2, 12, 140, 16, 1, state="both", **kw)
    _check_scan(_gen(6), torch.bfloat16, 2, 12, 20, 16, 1, **kw)


@pytest.mark.parametrize("L", [5000, 4096])
def test_scan_of_few_rows_over_a_long_axis(L):
    _check_scan(_gen(L), torch.float32, 1, 6, L, 16, 1, state="both")
    _check_scan(_gen(L), torch.bfloat16, 2, 3, L, 8, 1, lengths=[L, 2500], state="inplace")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [192, 320, 383, 384, 385, 512, 513])
def test_scan_lengths_around_whole_chunks(dtype, L):
    _check_scan(_gen(L), dtype, 2, 19, L, 16, state="both")
    _check_scan(_gen(L), dtype, 3, 18, L, 24, 2, lengths=[L, 129, 0], state="inplace", strided=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,G,D,L", [(24, 2, 40, 1100), (5, 1, 17, 769), (64, 1, 16, 1500), (239, 1, 4, 800), (256, 1, 4, 800)])
def test_scan_in_segments(dtype, N, G, D, L):
    _check_scan(_gen(N), dtype, 2, D, L, N, G, state="both", z=N != 5)
    _check_scan(_gen(N), dtype, 4, D, L, N, G, lengths=[L, 0, 1, L - 300], slots=[5, 1, -2, 0], pool=6, state="inplace",
                strided=True)


def test_scan_of_many_rows():
    """More workgroups than two a CU: nothing is read ahead."""
    _check_scan(_gen(17), torch.bfloat16, 40, 255, 300, 16, 1, lengths=[300] * 20 + list(range(20)), state="inplace")


def test_scan_large_steps_forget():
    """Steps so long that exp(s A) is 0 (and the product over a segment underflows): each output
    depends on its own position alone, and nothing becomes NaN."""
    g = _gen(8)
    s = _scan_inputs(g, torch.float32, 1, 4, 400, 16, 1)
    s["dt"].fill_(100.0)
    s["A"].fill_(-50.0)
    want, bound, _, _ = ref.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], True, None,
                                           None, None, None)
    out = sc.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    ref.assert_within(out, want, bound, "scan")


def test_scan_infinity_stays_where_it_is():
    """An infinite input makes its own channel's later outputs infinite or NaN, and no other's."""
    g = _gen(10)
    s = _scan_inputs(g, torch.float32, 2, 40, 300, 16, 1)
    clean = sc.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    s["x"][1, 7, 33] = float("inf")
    out = sc.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    assert not torch.isfinite(out[1, 7, 33:]).any()
    keep = torch.ones(2, 40, 300, dtype=torch.bool, device="cuda")
    keep[1, 7, 33:] = False
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,D,N,G,pool,slots", [(1, 1, 16, 1, None, None), (3, 37, 16, 1, None, None),
                                                (2, 34, 5, 2, None, None), (4, 130, 24, 1, 6, [5, 0, 3, 1]),
                                                (4, 66, 64, 3, 5, [4, -1, 99, 0]), (2, 7, 1, 1, None, None),
                                                (2, 9, 256, 1, None, None), (2, 20, 130, 2, None, None)])
def test_scan_step(dtype, B, D, N, G, pool, slots):
    g = _gen(B + D + N)
    s = _scan_inputs(g, dtype, B, 2 * D, 1, N, 2 * G)
    x, dt, z = (s[k][:, D:, 0] for k in ("x", "dt", "z"))
    Bm, Cm = (s[k][:, G:, :, 0] for k in ("B", "C"))
    A, skip, bias = s["A"][:D].contiguous(), s["D"][:D].contiguous(), s["dt_bias"][:D].contiguous()
    state = _randn(g, pool or B, D, N)
    want, bound, P, PB = ref.selective_scan(x[:, :, None], dt[:, :, None], A, Bm[..., None], Cm[..., None], skip,
                                            z[:, :, None], bias, True, None, slots, state, state)
    out = sc.selective_scan_step(x, state, dt, A, Bm, Cm, D=skip, z=z, dt_bias=bias,
                                 slots=None if slots is None else _ints(slots))
    ref.assert_within(out[:, :, None], want, bound, "scan step")
    ref.assert_within(state, P, PB, "scan step state")


def test_scan_steps_repeat_the_prompt():
    g = _gen(11)
    B, D, L, N = 2, 24, 21, 16
    s = _scan_inputs(g, torch.float32, B, D, L, N, 1)
    kw = dict(D=s["D"], dt_bias=s["dt_bias"])
    want, bound, P, PB = ref.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], True, None,
                                            None, None, torch.zeros(B, D, N))
    state = torch.zeros(B, D, N, device="cuda")
    steps = torch.stack([sc.selective_scan_step(s["x"][..., t], state, s["dt"][..., t], s["A"], s["B"][..., t],
                                                s["C"][..., t], z=s["z"][..., t], **kw) for t in range(L)], 2)
    ref.assert_within(steps, want, bound, "steps")
    ref.assert_within(state, P, PB, "state after the steps")
    state.zero_()
    parts = [sc.selective_scan(s["x"][..., i:j], s["dt"][..., i:j], s["A"], s["B"][..., i:j], s["C"][..., i:j],
                               z=s["z"][..., i:j], initial_state=state, final_state=state, **kw)
             for i, j in ((0, 8), (8, 9), (9, L))]
    ref.assert_within(torch.cat(parts, 2), want, bound, "chunks")
    ref.assert_within(state, P, PB, "state after the chunks")


# ---- adapters


def _check_adapter(g, dtype, B, C, M, L, R, n, index=None, scale=True, base="given", strided=False):
    x = _randn(g, B, C, L, dtype=dtype)
    down, up = _randn(g, n, R, C, dtype=dtype, scale=C ** -0.5), _randn(g, n, M, R, dtype=dtype, scale=R ** -0.5)
    sv = _randn(g, n) if scale else None
    bs = _randn(g, B, M, L, dtype=dtype) if base != "none" else None
    if index is None:
        index = torch.randint(0, n, (B,), generator=g, device="cuda").tolist()
    want, bound = ref.adapter(x, down, up, index, sv, bs)
    if strided:
        x, bs = _strided(x), _strided(bs) if bs is not None else None
    out = bs if base == "inplace" else torch.full((B, M, L), NAN, dtype=dtype, device="cuda")
    sc.adapter_apply(x, down, up, _ints(index), scale=sv, base=bs, out=out)
    ref.assert_within(out, want, bound, "adapter")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 33, 64, 65, 127, 130, 200])
def test_adapter_lengths(dtype, L):
    _check_adapter(_gen(L), dtype, 3, 70, 90, L, 16, 4)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("C,M,R", [(1, 1, 1), (3, 5, 2), (16, 16, 4), (31, 33, 7), (64, 48, 8), (65, 129, 24), (257, 100, 32),
                                   (96, 200, 64), (130, 70, 100), (200, 257, 128), (1024, 512, 16)])
@pytest.mark.parametrize("L", [1, 50])
def test_adapter_sizes(dtype, C, M, R, L):
    _check_adapter(_gen(C + L), dtype, 2, C, M, L, R, 3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [256, 512, 1024, 1601])
@pytest.mark.parametrize("R", [3, 16, 40])
def test_adapter_long_rows(dtype, L, R):
    """Four tiles of positions side by side, all of them there or the last set cut short."""
    _check_adapter(_gen(L + R), dtype, 2, 70, 100, L, R, 3, index=[1, -1] if R == 3 else [2, 0])
    _check_adapter(_gen(L), dtype, 1, 300, 65, L, R, 1, base="inplace", strided=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [1, 37])
def test_adapter_index_base_and_strides(dtype, L):
    g = _gen(L)
    _check_adapter(g, dtype, 6, 40, 50, L, 8, 3, index=[-1, 0, 2, 3, 1, -7])
    _check_adapter(g, dtype, 4, 40, 50, L, 8, 3, index=[-1, 0, 2, 2], base="none", scale=False)
    _check_adapter(g, dtype, 4, 40, 50, L, 8, 3, index=[1, -1, 2, 2], base="inplace")
    _check_adapter(g, dtype, 4, 41, 51, L, 8, 3, base="given", strided=True)
    _check_adapter(g, dtype, 4, 41, 51, L, 8, 3, base="inplace", strided=True)
    _check_adapter(g, dtype, 70, 33, 17, L, 5, 3)


def test_adapter_nan_of_one_position_stays_there():
    g = _gen(12)
    x, down, up = _randn(g, 2, 40, 50), _randn(g, 1, 8, 40), _randn(g, 1, 30, 8)
    idx = _ints([0, 0])
    clean = sc.adapter_apply(x, down, up, idx)
    x[1, 3, 20] = NAN
    out = sc.adapter_apply(x, down, up, idx)
    assert torch.isnan(out[1, :, 20]).all()
    out[1, :, 20] = clean[1, :, 20]
    assert torch.equal(out, clean)


# ---- streams, graphs, long offsets, refusals that need device tensors


def test_other_stream_and_given_workspace():
    g = _gen(13)
    s = _scan_inputs(g, torch.float32, 1, 64, 4096, 16, 1)
    x, down, up, idx = _randn(g, 2, 64, 96), _randn(g, 2, 8, 64), _randn(g, 2, 48, 8), _ints([1, 0])
    w = _randn(g, 64, 4)
    args = (s["x"], s["dt"], s["A"], s["B"], s["C"])
    want = [sc.selective_scan(*args), sc.adapter_apply(x, down, up, idx), sc.causal_conv(s["x"], w)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [sc.selective_scan(*args, stream=side), sc.adapter_apply(x, down, up, idx, stream=side.cuda_stream),
           sc.causal_conv(s["x"], w, stream=side)]
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    ws = torch.empty(sc.selective_scan_workspace(s["x"], s["A"], 1) + 16, dtype=torch.uint8, device="cuda")
    assert torch.equal(sc.selective_scan(*args, workspace=ws), want[0])


def test_graph_replays_equal_the_eager_calls():
    g = _gen(14)
    B, D, L, N, K = 2, 64, 600, 16, 4
    s = _scan_inputs(g, torch.bfloat16, B, D, L, N, 1)
    w, idx = _randn(g, D, K), _ints([1, -1])
    down, up = _randn(g, 2, 8, D, dtype=torch.bfloat16), _randn(g, 2, D, 8, dtype=torch.bfloat16)
    hs, cs = torch.zeros(B, D, N, device="cuda"), torch.zeros(B, D, K - 1, dtype=torch.bfloat16, device="cuda")

    def run():
        u = sc.causal_conv(s["x"], w, initial_state=cs, final_state=cs)
        u = sc.adapter_apply(u, down, up, idx, base=u)
        y = sc.selective_scan(u, s["dt"], s["A"], s["B"], s["C"], z=s["z"], initial_state=hs, final_state=hs)
        a = sc.causal_conv_step(y[:, :, 5], cs, w)
        return y, sc.selective_scan_step(a, hs, s["dt"][:, :, 0], s["A"], s["B"][..., 0], s["C"][..., 0])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for k in range(3):
        s["x"].copy_(_randn(g, B, D, L, dtype=torch.bfloat16))
        hs.normal_(generator=g)
        cs.normal_(generator=g)
        before = hs.clone(), cs.clone()
        eager = [t.clone() for t in run()]
        after = hs.clone(), cs.clone()
        hs.copy_(before[0]), cs.copy_(before[1])
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip([*eager, *after], [*outs, hs, cs]):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Batches more than 2^32 bytes (and 2^31 values) apart."""
    g = _gen(15)
    B, D, L, N, far = 2, 8, 40, 16, (1 << 31) + 64
    big = torch.empty(far + D * L, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(far + D * L, dtype=torch.bfloat16, device="cuda")
    s = _scan_inputs(g, torch.bfloat16, B, D, L, N, 1)
    x = big.as_strided((B, D, L), (far, L, 1))
    y = out.as_strided((B, D, L), (far, L, 1))
    x.copy_(s["x"])
    w = _randn(g, D, 4)
    sc.causal_conv(x, w, out=y)
    assert torch.equal(y, sc.causal_conv(s["x"], w))
    sc.selective_scan(x, s["dt"], s["A"], s["B"], s["C"], z=s["z"], out=y)
    assert torch.equal(y, sc.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], z=s["z"]))
    down, up = _randn(g, 1, 4, D, dtype=torch.bfloat16), _randn(g, 1, D, 4, dtype=torch.bfloat16)
    sc.adapter_apply(x, down, up, _ints([0, 0]), base=x, out=y)
    assert torch.equal(y, sc.adapter_apply(s["x"], down, up, _ints([0, 0]), base=s["x"]))
    # states whose slots are that far apart
    pool = torch.empty(far + D * N, dtype=torch.float32, device="cuda").as_strided((B, D, N), (far, N, 1))
    small = _randn(g, B, D, N)
    pool.copy_(small)
    a = sc.selective_scan_step(s["x"][..., 0], pool, s["dt"][..., 0], s["A"], s["B"][..., 0], s["C"][..., 0])
    b = sc.selective_scan_step(s["x"][..., 0], small, s["dt"][..., 0], s["A"], s["B"][..., 0], s["C"][..., 0])
    assert torch.equal(a, b) and torch.equal(pool, small)


def test_empty_batches():
    e = torch.empty(0, 8, 5, device="cuda")
    assert sc.causal_conv(e, torch.ones(8, 4, device="cuda")).shape == (0, 8, 5)
    bc = torch.empty(0, 1, 16, 5, device="cuda")
    assert sc.selective_scan(e, e, torch.ones(8, 16, device="cuda"), bc, bc).shape == (0, 8, 5)
    assert sc.adapter_apply(e, torch.ones(1, 2, 8, device="cuda"), torch.ones(1, 3, 2, device="cuda"),
                            _ints([])).shape == (0, 3, 5)


def test_broadcast_inputs():
    """A stride of 0 repeats an input: one sequence for the whole batch."""
    g = _gen(16)
    s = _scan_inputs(g, torch.float32, 3, 8, 50, 16, 1)
    one = {k: s[k][:1] for k in ("x", "dt", "B", "C")}
    rep = {k: v.expand(3, *v.shape[1:]) for k, v in one.items()}
    full = {k: v.contiguous() for k, v in rep.items()}
    w = _randn(g, 8, 4)
    assert torch.equal(sc.causal_conv(rep["x"], w), sc.causal_conv(full["x"], w))
    a, b = (sc.selective_scan(v["x"], v["dt"], s["A"], v["B"], v["C"]) for v in (rep, full))
    assert torch.equal(a, b)


def test_refusals_of_the_binding():
    x = torch.zeros(2, 8, 16, device="cuda")
    w = torch.zeros(8, 4, device="cuda")
    A, bc = torch.zeros(8, 4, device="cuda"), torch.zeros(2, 1, 4, 16, device="cuda")
    down, up, idx = torch.zeros(1, 2, 8, device="cuda"), torch.zeros(1, 3, 2, device="cuda"), _ints([0, 0])
    bad = [lambda: sc.causal_conv(x.double(), w), lambda: sc.causal_conv(x.cpu(), w), lambda: sc.causal_conv(x[0], w),
           lambda: sc.causal_conv(x, w.half()), lambda: sc.causal_conv(x, w[:4]), lambda: sc.causal_conv(x, w.cpu()),
           lambda: sc.causal_conv(x.transpose(1, 2).contiguous().transpose(1, 2), w),
           lambda: sc.causal_conv(x, w, lengths=torch.zeros(2, dtype=torch.int64, device="cuda")),
           lambda: sc.causal_conv(x, w, lengths=_ints([1])), lambda: sc.causal_conv(x, w, bias=torch.zeros(7, device="cuda")),
           lambda: sc.causal_conv(x, w, out=torch.zeros(2, 8, 15, device="cuda")),
           lambda: sc.causal_conv(x, w, initial_state=torch.zeros(2, 8, 4, device="cuda")),
           lambda: sc.causal_conv(x, w, initial_state=torch.zeros(3, 8, 3, device="cuda"),
                                  final_state=torch.zeros(2, 8, 3, device="cuda")),
           lambda: sc.causal_conv_step(x[:, :, 0], torch.zeros(2, 8, 3, device="cuda").half(), w),
           lambda: sc.selective_scan(x, x.half(), A, bc, bc), lambda: sc.selective_scan(x, x, A[:, :3].contiguous(), bc, bc),
           lambda: sc.selective_scan(x, x, A, bc[:, 0], bc), lambda: sc.selective_scan(x, x, A, bc, bc, z=x[:, :, :8]),
           lambda: sc.selective_scan(x, x, A, bc, bc, D=torch.zeros(7, device="cuda")),
           lambda: sc.adapter_apply(x, down, up[:, :, :1].contiguous(), idx),
           lambda: sc.adapter_apply(x, down, up, idx, base=torch.zeros(2, 4, 16, device="cuda")),
           lambda: sc.adapter_apply(x, down, up, idx[:1].contiguous()),
           lambda: sc.adapter_apply(x, down.transpose(1, 2), up, idx)]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    refused = [lambda: sc.causal_conv(x, torch.zeros(8, 9, device="cuda")), lambda: sc.causal_conv(x, w, out=x),
               lambda: sc.causal_conv(x, w, initial_state=torch.zeros(1, 8, 3, device="cuda")),
               lambda: sc.selective_scan(x, x, A, torch.zeros(2, 3, 4, 16, device="cuda"), torch.zeros(2, 3, 4, 16, device="cuda")),
               lambda: sc.selective_scan(x, x, A, bc, bc, out=x),
               lambda: sc.adapter_apply(x, torch.zeros(1, 129, 8, device="cuda"), torch.zeros(1, 3, 129, device="cuda"), idx),
               lambda: sc.causal_conv(x, w, out=torch.zeros(1, 8, 16, device="cuda").expand(2, 8, 16))]
    for f in refused:
        with pytest.raises(sc.SparseConvError):
            f()
