"""The pruned attention layer, the page pool and the stack of layers: projections, rotary positions, cache, attention, norms and adapters
together, against the same layers in float64, and single positions against prompts.

Tolerance, as for the state space layer: every operator is within its own bound (test_gpu_attention.py); through a layer errors of fp32
size pass matrices of unit scale, so a layer's outputs, of unit scale, are held to 2^-24 times the sum over its inner sizes (channels,
dims, positions: the terms of each stage's sums, each stage's error amplified by at most the next one's 1-norm, about
the root of its size).  Through a stack each layer's error passes the ones after it, whose norms keep the scale: the layers'
tolerances are added and amplified by the 1-norm, the root of the channels, of the layers that follow."""
import numpy as np
import pytest
import torch

import sequence_ref as ref
import sparse_weight_direct_amd as sc
import test_gpu_ssm as ssm
from sparse_weight_direct_amd.cache import PagePool
from sparse_weight_direct_amd.hybrid import AttentionLayer, HybridStack
from sparse_weight_direct_amd.ssm import Adapters, StateSpaceLayer

pytestmark = pytest.mark.gpu

C, L = ssm.C, ssm.L  # the channels and the prompt length of the state space layer's tests
H, G, D, T = 6, 2, 16, 120
TOL = 2.0 ** -24 * (C + D + T + H * D) * np.sqrt(H * D)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _weights(seed):
    rng = np.random.default_rng(seed)

    def pruned(m, c):
        return (rng.standard_normal((m, c)) * (rng.random((m, c)) < 0.3) / np.sqrt(0.3 * c)).astype(np.float32)

    return pruned((H + 2 * G) * D, C), pruned(C, H * D)


FREQS = 100.0 ** (-np.arange(D // 2) / (D // 2))


def _attention64(qkv_w, out_w, u, adapted=lambda which, y, x: y, window=0, prefix=0, cap=0.0):
    """One sequence (C, n) from its start: (C, n)."""
    n = u.shape[1]
    qkv = adapted("in", qkv_w.astype(np.float64) @ u, u).reshape(H + 2 * G, D, n)
    t = np.arange(n)[None] * FREQS[:, None]
    a, b = qkv[:H + G, :D // 2], qkv[:H + G, D // 2:]
    turned = np.concatenate([a * np.cos(t) - b * np.sin(t), b * np.cos(t) + a * np.sin(t)], 1)
    i, j = np.arange(n)[:, None], np.arange(n)[None]
    seen = (j <= i) & ((i - j < window) if window else True) | (j < prefix)
    y = np.zeros((H, D, n))
    for h in range(H):
        g = h // (H // G)
        s = turned[h].T @ turned[H + g] * D ** -0.5
        if cap:
            s = cap * np.tanh(s / cap)
        s = np.where(seen, s, -np.inf)
        p = np.exp(s - s.max(1, keepdims=True))
        y[h] = qkv[H + G + g] @ (p / p.sum(1, keepdims=True)).T
    y = y.reshape(H * D, n)
    return adapted("out", out_w.astype(np.float64) @ y, y)


def _layer(pool, seed=0, layer=0, **kw):
    w = _weights(seed)
    return w, AttentionLayer(*w, pool, layer, length=L, freqs=torch.tensor(FREQS, dtype=torch.float64, device="cuda"), **kw)


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("kw", [dict(), dict(window=25), dict(cap=2.0)])
def test_prompts_and_single_positions(kw):
    """Prompts of unequal length in two chunks, then single positions, with adapters, against whole sequences in float64."""
    pool = PagePool(2, 60, G, D, page_size=16)
    w, m = _layer(pool, layer=1, **kw)
    g = _randn(5, 3, 4, C)
    ad = Adapters((g / 7, _randn(6, 3, (H + 2 * G) * D, 4) / 2, _randn(7, 3)), (_randn(8, 3, 4, H * D) / 10, _randn(9, 3, C, 4) / 2, None))
    index, split = [2, -1, 0], [(L, 30), (1, L), (7, 0)]
    ids = [pool.add() for _ in index]
    total = [a + b + 6 for a, b in split]
    u = _randn(1, 3, C, max(total))
    got = [[] for _ in ids]
    for part in range(2):
        n = [s[part] for s in split]
        chunk = torch.full((3, C, L), float("nan"), device="cuda")
        for i, k in enumerate(n):
            start = sum(split[i][:part])
            chunk[i, :, :k] = u[i, :, start:start + k]
            chunk[i, :, k:] = 0.0
        table, past = pool.extend(ids, n)
        out = m.prompt(chunk, table, past, _ints(n), adapters=ad, index=_ints(index))
        for i, k in enumerate(n):
            got[i].append(out[i, :, :k])
    for k in range(6):
        table, past = pool.extend(ids, [1, 1, 1])
        now = torch.stack([u[i, :, sum(split[i]) + k] for i in range(3)])
        out = m.step(now, table, past, adapters=ad, index=_ints(index))
        for i in range(3):
            got[i].append(out[i, :, None])
    for i in range(3):
        r = index[i]

        def adapted(which, y, x):
            down, up, scale = ad.in_proj if which == "in" else ad.out_proj
            return y if r < 0 else y + (1.0 if scale is None else float(scale[r])) * (ref.f64(up[r]) @ (ref.f64(down[r]) @ x))

        want = _attention64(*w, ref.f64(u[i, :, :total[i]]), adapted, **kw)
        assert np.abs(ref.f64(torch.cat(got[i], 1)) - want).max() <= TOL, i


def test_prefix_and_given_positions():
    pool = PagePool(1, 20, G, D, page_size=16)
    w, m = _layer(pool)
    u = _randn(2, 2, C, L)
    ids = [pool.add(), pool.add()]
    table, past = pool.extend(ids, [L, L], width=5)
    place = torch.arange(L, dtype=torch.int32, device="cuda").expand(2, 1, L).contiguous()
    out = m.prompt(u, table, past, positions=place, prefix=_ints([20, 0]))
    for i, p in enumerate((20, 0)):
        assert np.abs(ref.f64(out[i]) - _attention64(*w, ref.f64(u[i]), prefix=p)).max() <= TOL


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_forks_share_pages_until_they_differ(dtype):
    """Two branches of one prompt, and the same positions in sequences of their own: the same bits."""
    pool = PagePool(1, 40, G, D, page_size=16, dtype=dtype)
    w, m = _layer(pool)
    u, tail = _randn(3, 1, C, L), _randn(4, 5, 2, C)
    a, c, d = pool.add(), pool.add(), pool.add()
    table, past = pool.extend([a, c, d], [L - 3] * 3)
    first = m.prompt(u.expand(3, C, L).contiguous(), table, past, _ints([L - 3] * 3))
    assert torch.equal(first[0], first[1]) and torch.equal(first[0], first[2])
    free = pool.free_pages
    b = pool.fork(a)
    assert pool.free_pages == free
    for k in range(5):
        table, past = pool.extend([a, b, c, d], [1] * 4)
        x = tail[k][[0, 1, 0, 1]]
        y = m.step(x, table, past)
        assert torch.equal(y[0], y[2]) and torch.equal(y[1], y[3]) and not torch.equal(y[0], y[1])
        if k == 2:
            pool.free(pool.add())
            used = pool.compact()
            assert used == pool.pages - pool.free_pages
    pool.free(a)
    table, past = pool.extend([b, d], [1, 1])
    y = m.step(tail[0][[0, 0]], table, past)
    assert torch.equal(y[0], y[1])


def test_windows_give_their_pages_back():
    pool = PagePool(1, 12, G, D, page_size=16)
    w, m = _layer(pool, window=20)
    u = _randn(3, 1, C, L + 40)
    a = pool.add()
    table, past = pool.extend([a], [L])
    m.prompt(u[:, :, :L].contiguous(), table, past)
    want = _attention64(*w, ref.f64(u[0]), window=20)
    for k in range(40):
        table, past = pool.extend([a], [1])
        y = m.step(u[:, :, L + k].contiguous(), table, past)
        assert np.abs(ref.f64(y[0]) - want[:, L + k]).max() <= TOL, k
        pool.forget(a, L + k + 1 - 19)  # what the next position's window has passed
    assert (pool.table([a]) < 0).sum() == 3 and pool.free_pages == 12 - 2


def _stack(seed=0):
    host, dev, _, _ = ssm._weights(seed)
    pool = PagePool(2, 40, G, D, page_size=16)
    w0, a0 = _layer(pool, seed=seed + 1, layer=0)
    w1, a1 = _layer(pool, seed=seed + 2, layer=1, window=30)
    s = StateSpaceLayer(host["in_proj"], host["x_proj"], host["dt_proj"], host["out_proj"], **dev, length=L, slots=4)
    weights, post = 1.0 + _randn(seed + 3, 4, C) / 10, 1.0 + _randn(seed + 4, 3, C) / 10

    def want(x, n):
        def norm(v, w):
            return v / np.sqrt((v * v).mean(0, keepdims=True) + 1e-6) * ref.f64(w)[:, None]

        r = ref.f64(x)[:, :n]
        h = norm(r, weights[0])
        calls = [lambda h: _attention64(*w0, h), lambda h: ssm._reference(host, dev, Adapters(), torch.tensor(h)[None], [n], [-1])[0],
                 lambda h: _attention64(*w1, h, window=30)]
        for i, call in enumerate(calls):
            r = r + 0.5 * norm(call(h), post[i])
            h = norm(r, weights[i + 1])
        return h

    return pool, HybridStack([a0, s, a1], weights, post_weights=post, scale=0.5), want


TOL_STACK = (2 * TOL + ssm.TOL) * np.sqrt(C)


def test_stack_of_attending_and_scanning_layers():
    pool, stack, want = _stack()
    x = _randn(11, 3, C, L + 8)
    x0 = x.clone()
    n, ids, slots = [L, 5, 21], [pool.add() for _ in range(3)], _ints([2, 0, 3])
    table, past = pool.extend(ids, n)
    out = stack.prompt(x[:, :, :L].contiguous(), slots, table, past, _ints(n))
    full = [want(x[i], k + 8) for i, k in enumerate(n)]
    for i, k in enumerate(n):
        assert np.abs(ref.f64(out[i, :, :k]) - full[i][:, :k]).max() <= TOL_STACK, i
    for j in range(8):
        table, past = pool.extend(ids, [1] * 3)
        y = stack.step(torch.stack([x[i, :, k + j] for i, k in enumerate(n)]), slots, table, past)
        for i, k in enumerate(n):
            assert np.abs(ref.f64(y[i]) - full[i][:, k + j]).max() <= TOL_STACK, (i, j)
    assert torch.equal(x, x0)


def test_stack_steps_replayed_from_a_graph():
    """A captured step with its position advanced inside, replayed with eager work between, against eager steps."""
    pool, stack, _ = _stack(3)
    other, eager, _ = _stack(3)
    x, slots = _randn(5, 2, C, L), _ints([1, 3])
    for p, s in ((pool, stack), (other, eager)):
        ids = [p.add(), p.add()]
        table, past = p.extend(ids, [L, L - 9], width=6)
        s.prompt(x, slots, table, past, _ints([L, L - 9]))
    table, past = pool.extend([0, 1], [12, 12], width=6)
    now = _randn(6, 2, C)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    state = stack.layers[1].conv_state.clone(), stack.layers[1].scan_state.clone()
    with torch.cuda.stream(side):
        stack.step(now, slots, table, past)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = stack.step(now, slots, table, past)
        past.add_(1)
    stack.layers[1].conv_state.copy_(state[0])
    stack.layers[1].scan_state.copy_(state[1])
    for k in range(6):
        now.copy_(_randn(20 + k, 2, C))
        graph.replay()
        t, p = other.extend([0, 1], [1, 1], width=6)
        want = eager.step(now, slots, t, p)
        torch.cuda.synchronize()
        assert torch.equal(out, want), k


def test_refusals_of_the_layers():
    pool = PagePool(1, 10, G, D, page_size=16)
    w, m = _layer(pool)
    a = pool.add()
    table, past = pool.extend([a], [3])
    for bad in (_randn(0, 1, C, L + 1), _randn(0, 1, C + 1, L), _randn(0, 1, C)):
        with pytest.raises(ValueError):
            m.prompt(bad, table, past)
    with pytest.raises(ValueError):
        m.step(_randn(0, 1, C, 1), table, past)
    with pytest.raises(ValueError):
        m.step(_randn(0, 2, C), table, past)
    for args in ((w[0][:-1], w[1]), (w[0], w[1][:, :-1]), (w[0][:2 * G * D], w[1]), (w[0][:(2 * G + 1) * D], w[1])):
        with pytest.raises(ValueError):
            AttentionLayer(*args, pool, 0, length=L)
    with pytest.raises(ValueError):
        AttentionLayer(*w, pool, 1, length=L)
    for bad in (torch.ones(3, C, device="cuda"), torch.ones(2, C), torch.ones(2, C, dtype=torch.float64, device="cuda")):
        with pytest.raises(ValueError):
            HybridStack([m], bad)
    with pytest.raises(ValueError):
        HybridStack([m, AttentionLayer(*w, pool, 0, length=L + 1)], torch.ones(3, C, device="cuda"))
