"""The attention operators where calls meet: other streams and given workspaces, graphs, offsets past 32 bits, refusals, gradients,
versions, and every kernel that only large calls take."""
import pytest
import torch

import attention_ref as ref
import sparse_weight_direct_amd as sc
from test_gpu_attention import INF, NAN, TYPES, _cache, _check, _check_append, _check_norm, _gen, _ints, _randn

pytestmark = pytest.mark.gpu


def test_other_streams_and_given_workspaces():
    """Two calls at once on two streams, each with its workspace, and the same on the stream's handle."""
    g = _gen(1)
    k, v, table = _cache(g, torch.bfloat16, 2, 128, 64, [5000, 3000], None, 1)
    q = _randn(g, 2, 8 * 128, dtype=torch.bfloat16)
    past = _ints([5000, 3000])
    want = sc.paged_attention_step(q, k, v, table, past)
    need = sc.paged_attention_workspace(2, 8, 1, k, table.shape[1])
    assert need > 0
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [sc.paged_attention_step(q, k, v, table, past, stream=s, workspace=w) for s, w in zip(streams, spaces)]
        got.append(sc.paged_attention_step(q, k, v, table, past, stream=streams[0].cuda_stream, workspace=spaces[0]))
        with torch.cuda.stream(streams[1]):
            got.append(sc.paged_attention_step(q, k, v, table, past))
        torch.cuda.synchronize()
        assert all(torch.equal(x, want) for x in got)
    with pytest.raises(sc.SparseConvError):
        sc.paged_attention_step(q, k, v, table, past, workspace=spaces[0][:need - 256])
    x, y = _randn(g, 2, 64, 40), _randn(g, 2, 64, 40)
    w = torch.ones(64, device="cuda")
    want = sc.residual_norm(x, y, weight=w)
    torch.cuda.synchronize()
    got = sc.residual_norm(x, y, weight=w, stream=streams[0])
    pool = _randn(g, 3, 9, 64)
    expected = pool.clone()
    expected[:, 4] = pool[:, 2]
    a = _ints([2]), _ints([4])
    torch.cuda.synchronize()
    sc.cache_copy(pool, *a, stream=streams[1])
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(pool, expected)


def test_graph_replays_equal_the_eager_calls():
    g = _gen(2)
    past = _ints([700, 0, 31, 2000])
    k, v, table = _cache(g, torch.bfloat16, 2, 64, 16, [700, 0, 31, 2000], None, 8)
    k, v = torch.nan_to_num(k), torch.nan_to_num(v)
    qkv, x, w = _randn(g, 4, 12 * 64, dtype=torch.bfloat16), _randn(g, 4, 256, dtype=torch.bfloat16), _randn(g, 256)
    freqs = torch.pow(100.0, -torch.arange(32, device="cuda", dtype=torch.float64) / 32)
    pool = torch.stack([k.flatten(1), v.flatten(1)])
    kp, vp = pool[0].view(k.shape), pool[1].view(v.shape)
    source, target = _ints([int(table[0, 0])]), _ints([int(table[1, 3])])  # (nobody reads that one)

    def call():
        r, h = sc.residual_norm_step(x, x.clone(), weight=w, post_weight=w)
        q = sc.cache_append_step(qkv[:, 512:640], qkv[:, 640:], kp, vp, table, past, q=qkv[:, :512], freqs=freqs)
        o = sc.paged_attention_step(q, kp, vp, table, past)
        sc.cache_copy(pool, source, target)
        return r, h, q, o

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for i in range(5):
        qkv.copy_(_randn(g, 4, 12 * 64, dtype=torch.bfloat16))
        x.copy_(_randn(g, 4, 256, dtype=torch.bfloat16))
        past.add_(1)
        before = pool.clone()
        want = [t.clone() for t in call()]
        after = pool.clone()
        pool.copy_(before)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(pool, after), i


def test_offsets_past_32_bits():
    """Pages whose offsets pass 2^31 values and 2^32 bytes, and a batch stride past both."""
    g = _gen(3)
    G, P, D, pages = 8, 256, 128, 8300  # 2.2 * 2^31 bytes of keys in 16 bits: 2^31 values and more
    per = G * P * D
    assert pages * per > 2 ** 31
    k = torch.zeros(pages, G, P, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros(pages, G, D, P, dtype=torch.bfloat16, device="cuda")
    table = _ints([[pages - 1, 3], [8200, pages - 2]])
    past = _ints([300, 200])
    kk, vv, q = _randn(g, 2, G * D, 90, dtype=torch.bfloat16), _randn(g, 2, G * D, 90, dtype=torch.bfloat16), _randn(g, 2, 16 * D, 90, dtype=torch.bfloat16)
    small = _ints([[0, 1], [2, 3]])
    for t in table.flatten().tolist():
        k[t] = _randn(g, G, P, D, dtype=torch.bfloat16)
        v[t] = _randn(g, G, D, P, dtype=torch.bfloat16)
    ks, vs = k[table.flatten().long()].clone(), v[table.flatten().long()].clone()
    a = sc.cache_append(kk, vv, k, v, table, past, q=q)
    b = sc.cache_append(kk, vv, ks, vs, small, past, q=q)
    assert torch.equal(a, b) and torch.equal(k[table.flatten().long()], ks) and torch.equal(v[table.flatten().long()], vs)
    for n in (1, 90):
        x = q[:, :, :n].contiguous()
        assert torch.equal(sc.paged_attention(x, k, v, table, past), sc.paged_attention(x, ks, vs, small, past))
    pool = k.view(1, pages, per)
    sc.cache_copy(pool, _ints([pages - 1]), _ints([8201]))
    assert torch.equal(k[8201], k[pages - 1])
    x = torch.empty(2, 16, 2 ** 26 + 9, dtype=torch.bfloat16, device="cuda")[:, :, -70:]  # batches 2^30 values, 2^31 bytes apart
    x.copy_(_randn(g, 2, 16, 70))
    w = torch.ones(16, device="cuda")
    assert torch.equal(sc.residual_norm(x, x.contiguous(), weight=w)[1], sc.residual_norm(x.contiguous(), x.contiguous(), weight=w)[1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 80, 128, 192, 256])
def test_many_rows_of_every_width(dtype, D):
    """The kernel whose wavefronts share the keys, for whole and partial widths, whole and split contexts, small and large pages."""
    g = _gen(D)
    _check(g, dtype, 1, 4, 1, D, 70, 16, [200])
    _check(g, dtype, 1, 2, 1, D, 130, 64, [1000], extra=30)
    _check(g, dtype, 2, 2, 2, D, 140, 256, [0, 60], lengths=[140, 129], window=50, prefix=[5, 0], cap=8.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_few_rows_in_two_and_four_tiles(dtype):
    g = _gen(17)
    for L in (5, 9, 12, 16):  # with four heads a head of keys: 20 to 64 rows
        for D in (64, 128, 256):
            _check(g, dtype, 1, 4, 1, D, L, 64, [130], window=77)


def test_kernels_of_the_norms_that_sizes_choose():
    g = _gen(5)
    for C, L in ((1000, 2050), (2048, 1100), (500, 4100)):  # two tiles for every CU
        _check_norm(g, torch.bfloat16, 8, C, L, gate="channels")
    for C in (3000, 4096, 8192, 8193):
        for dtype in (torch.float32, torch.float16):
            _check_norm(g, dtype, 2, C, 1, gate="all", center=True)
            _check_norm(g, dtype, 1, C, 37, gate="all")


def test_append_of_many_heads_and_tiles():
    g = _gen(6)
    _check_append(g, torch.bfloat16, torch.bfloat16, 4, 20, 4, 64, 400, 64, [0, 70, 5, 300], axes=3)
    _check_append(g, torch.float32, torch.float16, 2, 33, 3, 128, 700, 128, [3, 64], lengths=[700, 1], pairs=40)
    _check_append(g, torch.float32, torch.float32, 1, 9, 9, 256, 130, 16, [11], interleaved=True)


def test_a_fork_is_copied_before_its_next_positions():
    """A run of the operators as they are used: append, fork by a copy, append to both, attend to both."""
    g = _gen(7)
    for dtype in TYPES:
        G, D, P, pages = 2, 64, 32, 12
        pool = torch.full((2, pages, G * P * D), NAN, dtype=dtype, device="cuda")
        kp, vp = pool[0].view(pages, G, P, D), pool[1].view(pages, G, D, P)
        freqs = torch.pow(1000.0, -torch.arange(D // 2, device="cuda", dtype=torch.float64) / (D // 2))
        qkv = [_randn(g, 1, n * D, 50, dtype=dtype) for n in (4, G, G)]
        table = _ints([[7, 2, 9]])
        sc.cache_append(qkv[1], qkv[2], kp, vp, table, _ints([0]), q=qkv[0], freqs=freqs)
        sc.cache_copy(pool, _ints([2]), _ints([5]))
        both = _ints([[7, 2, 9], [7, 5, 11]])
        more = [_randn(g, 2, n * D, 30, dtype=dtype) for n in (4, G, G)]
        q = sc.cache_append(more[1], more[2], kp, vp, both, _ints([50, 50]), q=more[0], freqs=freqs)
        out = sc.paged_attention(q, kp, vp, both, _ints([50, 50]))
        ref.check_attention(out, ref.paged_attention(q, kp, vp, both, _ints([50, 50])))
        for b in range(2):  # each as if it had been alone
            k1, v1 = torch.full_like(kp, NAN), torch.full_like(vp, NAN)
            sc.cache_append(qkv[1], qkv[2], k1, v1, table, _ints([0]), freqs=freqs)
            q1 = sc.cache_append(more[1][b:b + 1], more[2][b:b + 1], k1, v1, table, _ints([50]), q=more[0][b:b + 1], freqs=freqs)
            assert torch.equal(q1[0], q[b]) and torch.equal(sc.paged_attention(q1, k1, v1, table, _ints([50]))[0], out[b])


def test_chunks_equal_their_single_positions():
    """What a chunk gives is what its positions give one by one, to the kernels' rounding."""
    g = _gen(8)
    k, v, table = _cache(g, torch.float32, 2, 64, 32, [100], None, 6)
    q = _randn(g, 1, 4 * 64, 6)
    chunk = sc.paged_attention(q, k, v, table, _ints([100]))
    for i in range(6):
        one = sc.paged_attention_step(q[:, :, i], k, v, table, _ints([100 + i]))
        want = ref.paged_attention(q[:, :, i:i + 1], k, v, table, _ints([100 + i]))
        ref.check_attention(one[:, :, None], want)
        assert ((chunk[:, :, i] - one).abs().cpu().double() <= 2 * want[1][:, :, 0]).all()


def test_an_infinite_query_spoils_its_own_row():
    g = _gen(9)
    for L in (6, 150):
        k, v, table = _cache(g, torch.bfloat16, 1, 64, 32, [40], None, L)
        q = _randn(g, 1, 128, L, dtype=torch.bfloat16)
        want = ref.paged_attention(q, k, v, table, _ints([40]))
        bad = q.clone()
        bad[0, 3, 2], bad[0, 70, 4] = INF, NAN
        got = ref.wide(sc.paged_attention(bad, k, v, table, _ints([40]))).view(1, 2, 64, L)
        keep = torch.ones(1, 2, 64, L, dtype=torch.bool)
        keep[0, 0, :, 2] = keep[0, 1, :, 4] = False
        out, bound = want[0].view(1, 2, 64, L), want[1].view(1, 2, 64, L)
        assert torch.isfinite(got[keep]).all() and ((got - out).abs() <= bound)[keep].all()
        assert torch.isnan(got[0, 1, :, 4]).all()


REFUSED = [
    ("paged_attention", lambda t: dict(q=t["q"][0])), ("paged_attention", lambda t: dict(q=t["q"].double())),
    ("paged_attention", lambda t: dict(q=t["q"].cpu())), ("paged_attention", lambda t: dict(q=t["q"][:, :-1])),
    ("paged_attention", lambda t: dict(q=t["q"].transpose(1, 2).contiguous().transpose(1, 2))),
    ("paged_attention", lambda t: dict(k_pages=t["k_pages"].half())), ("paged_attention", lambda t: dict(k_pages=t["k_pages"].transpose(2, 3))),
    ("paged_attention", lambda t: dict(v_pages=t["v_pages"][:-1])), ("paged_attention", lambda t: dict(v_pages=t["k_pages"][:, :, :8])),
    ("paged_attention", lambda t: dict(table=t["table"].long())), ("paged_attention", lambda t: dict(table=t["table"][:1])),
    ("paged_attention", lambda t: dict(table=t["table"].t().contiguous().t())), ("paged_attention", lambda t: dict(past=t["past"][:1])),
    ("paged_attention", lambda t: dict(past=t["past"].long())), ("paged_attention", lambda t: dict(past=None)),
    ("paged_attention", lambda t: dict(lengths=t["past"].float())), ("paged_attention", lambda t: dict(slopes=torch.ones(3, device="cuda"))),
    ("paged_attention", lambda t: dict(prefix=t["past"][:1])), ("paged_attention", lambda t: dict(window=-1)),
    ("paged_attention", lambda t: dict(scale="x")), ("paged_attention", lambda t: dict(cap=-1.0)), ("paged_attention", lambda t: dict(scale=NAN)),
    ("paged_attention", lambda t: dict(out=t["q"].half())), ("paged_attention", lambda t: dict(out=t["q"])),
    ("cache_append", lambda t: dict(k=t["k"][:, :-1])), ("cache_append", lambda t: dict(v=t["v"][:1])), ("cache_append", lambda t: dict(v=t["v"].half())),
    ("cache_append", lambda t: dict(k=t["k"].half(), v=t["v"].half())), ("cache_append", lambda t: dict(q=t["q"][:, :-1])),
    ("cache_append", lambda t: dict(freqs=t["freqs"].float())), ("cache_append", lambda t: dict(freqs=t["freqs"].repeat(3))),
    ("cache_append", lambda t: dict(axes=t["axes"][:-1])), ("cache_append", lambda t: dict(positions=t["positions"][:, 0])),
    ("cache_append", lambda t: dict(positions=t["positions"][:, :, :-1])), ("cache_append", lambda t: dict(freqs=None)),
    ("cache_append", lambda t: dict(q=None, out=t["q"])), ("cache_append", lambda t: dict(out=t["q"].half())),
    ("cache_append", lambda t: dict(out=t["q"][:, :48])), ("cache_append", lambda t: dict(v_pages=t["k_pages"].view(t["v_pages"].shape))),
    ("cache_copy", lambda t: dict(pool=t["pool"][0])), ("cache_copy", lambda t: dict(pool=t["pool"].cpu())),
    ("cache_copy", lambda t: dict(pool=t["pool"].transpose(1, 2))), ("cache_copy", lambda t: dict(source=t["source"].long())),
    ("cache_copy", lambda t: dict(source=t["source"][:1])), ("cache_copy", lambda t: dict(target=t["source"].cpu())),
    ("cache_copy", lambda t: dict(pool=t["pool"][:, :1].expand(2, 9, 64))),
    ("residual_norm", lambda t: dict(x=t["x"][0])), ("residual_norm", lambda t: dict(y=t["y"][:, :-1])), ("residual_norm", lambda t: dict(y=t["y"].half())),
    ("residual_norm", lambda t: dict(weight=t["w"][:-1])), ("residual_norm", lambda t: dict(weight=t["w"].half())),
    ("residual_norm", lambda t: dict(gate=t["y"][:, :, :-1])), ("residual_norm", lambda t: dict(y=None)),
    ("residual_norm", lambda t: dict(weight=None, bias=t["w"])), ("residual_norm", lambda t: dict(eps=-1.0)),
    ("residual_norm", lambda t: dict(scale=None)), ("residual_norm", lambda t: dict(sum=t["y"])), ("residual_norm", lambda t: dict(out=t["x"])),
    ("residual_norm", lambda t: dict(out=t["x"], sum=t["x"])), ("residual_norm", lambda t: dict(weight=None, post_bias=t["w"])),
]


def _tensors():
    g = _gen(10)
    k, v, table = _cache(g, torch.float32, 2, 16, 16, [5, 20], None, 12)
    pool = _randn(g, 2, 9, 64)
    x = _randn(g, 2, 64, 12)
    return dict(q=_randn(g, 2, 64, 12), k=_randn(g, 2, 32, 12), v=_randn(g, 2, 32, 12), k_pages=k, v_pages=v, table=table, past=_ints([5, 20]),
                freqs=torch.ones(8, dtype=torch.float64, device="cuda"), axes=_ints([0] * 8), positions=torch.zeros(2, 1, 12, dtype=torch.int32, device="cuda"),
                pool=pool, source=_ints([1, 2]), target=_ints([3, 4]), x=x, y=_randn(g, 2, 64, 12), w=_randn(g, 64))


def _arguments(t, name):
    if name == "paged_attention":
        return dict(q=t["q"], k_pages=t["k_pages"], v_pages=t["v_pages"], table=t["table"], past=t["past"])
    if name == "cache_append":
        return dict(k=t["k"], v=t["v"], k_pages=t["k_pages"], v_pages=t["v_pages"], table=t["table"], past=t["past"], q=t["q"], freqs=t["freqs"],
                    axes=t["axes"], positions=t["positions"])
    if name == "cache_copy":
        return dict(pool=t["pool"], source=t["source"], target=t["target"])
    return dict(x=t["x"], y=t["y"], weight=t["w"], gate=t["y"])


@pytest.mark.parametrize("case", range(len(REFUSED)))
def test_refusals_of_the_binding(case):
    name, change = REFUSED[case]
    t = _tensors()
    kept = {n: x.clone() for n, x in t.items()}
    a = _arguments(t, name)
    getattr(sc, name)(**a)  # as it is it runs
    for n, x in t.items():
        x.copy_(kept[n])
    with pytest.raises((ValueError, sc.SparseConvError)) as e:
        getattr(sc, name)(**{**a, **change(t)})
    assert str(e.value)
    torch.cuda.synchronize()
    assert all(torch.equal(torch.nan_to_num(x.float()), torch.nan_to_num(kept[n].float())) for n, x in t.items())


@pytest.mark.parametrize("name", ["paged_attention", "cache_append", "cache_copy", "residual_norm"])
def test_tensors_that_require_gradients_are_refused(name):
    t = _tensors()
    a = _arguments(t, name)
    for n, x in a.items():
        if x.is_floating_point():
            b = {**a, n: x.detach().clone().requires_grad_()}
            with pytest.raises(ValueError, match="gradient"):
                getattr(sc, name)(**b)
            with torch.no_grad():
                getattr(sc, name)(**b)


def test_tensors_written_in_place_count_their_versions():
    t = _tensors()
    def counts(f, *tensors):
        before = [x._version for x in tensors]
        f()
        return [x._version - n for x, n in zip(tensors, before)]

    out = torch.empty_like(t["q"])
    assert counts(lambda: sc.paged_attention(**_arguments(t, "paged_attention"), out=out), out, t["q"], t["k_pages"]) == [1, 0, 0]
    assert counts(lambda: sc.cache_append(**_arguments(t, "cache_append"), out=out), out, t["k_pages"], t["v_pages"], t["q"]) == [1, 1, 1, 0]
    assert counts(lambda: sc.cache_append(**_arguments(t, "cache_append")), t["k_pages"], t["v_pages"], t["k"]) == [1, 1, 0]
    assert counts(lambda: sc.cache_copy(**_arguments(t, "cache_copy")), t["pool"], t["source"]) == [1, 0]
    s, o = torch.empty_like(t["x"]), torch.empty_like(t["x"])
    assert counts(lambda: sc.residual_norm(**_arguments(t, "residual_norm"), sum=s, out=o), s, o, t["x"], t["y"]) == [1, 1, 0, 0]


def test_empty_pools_are_refused():
    t = _tensors()
    with pytest.raises(sc.SparseConvError):
        sc.paged_attention(t["q"], t["k_pages"][:0], t["v_pages"][:0], t["table"], t["past"])
    with pytest.raises(sc.SparseConvError):
        sc.cache_append(t["k"], t["v"], t["k_pages"][:0], t["v_pages"][:0], t["table"], t["past"])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [16, 17, 32, 33, 95, 96])
def test_rows_where_the_kernel_changes(dtype, D, rows):
    g = _gen(D + rows)
    _check(g, dtype, 2, rows, 1, D, 1, 32, [700, 0])
    _check(g, dtype, 2, 1, 1, D, rows, 64, [40, 333], lengths=[rows, rows - 9], window=50, prefix=[70, 0])
