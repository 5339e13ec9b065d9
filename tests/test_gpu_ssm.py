"""The pruned state space layer: projections, convolution, scan and adapters together, against the
same layer in float64, and its single positions against its prompts.

Tolerance: every operator is within its own bound (test_gpu_sequence.py, test_gpu_parity.py); through
the layer errors of fp32 size pass five products of unit-scale matrices, so the outputs, of unit
scale, are held to 2^-24 times the sum over the layer's inner sizes (C + 2 D + R + N terms a value at
each stage, each stage's error amplified by at most the next one's 1-norm, about sqrt of its size)."""
import numpy as np
import pytest
import torch

import sequence_ref as ref
from sparse_weight_direct_amd.ssm import Adapters, StateSpaceLayer

pytestmark = pytest.mark.gpu

C, D, N, R, K, L, SLOTS = 48, 96, 16, 8, 4, 40, 6
TOL = 2.0 ** -24 * (C + 2 * D + R + N) * np.sqrt(D)


def _weights(seed=0):
    rng = np.random.default_rng(seed)

    def pruned(m, c):
        return (rng.standard_normal((m, c)) * (rng.random((m, c)) < 0.3) / np.sqrt(0.3 * c)).astype(np.float32)

    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*s):
        return torch.randn(s, generator=g, device="cuda")

    host = dict(in_proj=pruned(2 * D, C), x_proj=pruned(R + 2 * N, D), dt_proj=pruned(D, R), out_proj=pruned(C, D))
    dev = dict(conv_weight=r(D, K) / 2, conv_bias=r(D) / 10, A=-torch.exp(r(D, N) / 2), skip=r(D), dt_bias=r(D) - 2)
    ad = Adapters((r(3, 4, C) / 7, r(3, 2 * D, 4) / 2, r(3)), (r(3, 4, D) / 10, r(3, C, 4) / 2, None))
    return host, dev, ad, r


def _reference(host, dev, ad, u, lengths, index):
    """The layer on sequences that start anew: values alone, float64."""
    w = {k: v.astype(np.float64) for k, v in host.items()}
    U = ref.f64(u)
    out = np.zeros_like(U)
    for i in range(U.shape[0]):
        n, r = int(lengths[i]), int(index[i])

        def adapted(which, y, x):
            if which is None or not 0 <= r < which[0].shape[0]:
                return y
            s = 1.0 if which[2] is None else float(which[2][r])
            return y + s * (ref.f64(which[1][r]) @ (ref.f64(which[0][r]) @ x))

        x0 = U[i, :, :n]
        xz = adapted(ad.in_proj, w["in_proj"] @ x0, x0)

        dv = {k: v.double() for k, v in dev.items()}
        v = _conv64(xz[:D], dv)
        p = w["x_proj"] @ v
        y = _scan64(v, w["dt_proj"] @ p[:R], p[R:R + N], p[R + N:], xz[D:], dv)
        out[i, :, :n] = adapted(ad.out_proj, w["out_proj"] @ y, y)
    return out


def _conv64(x, dv):
    w, b = ref.f64(dv["conv_weight"]), ref.f64(dv["conv_bias"])
    u = np.concatenate([np.zeros((D, K - 1)), x], 1)
    v = b[:, None] + sum(w[:, k, None] * u[:, k:k + x.shape[1]] for k in range(K))
    return v * ref.sigmoid(v)


def _scan64(x, dt, b, c, z, dv):
    A, skip, bias = (ref.f64(dv[k]) for k in ("A", "skip", "dt_bias"))
    s = np.logaddexp(0.0, dt + bias[:, None])
    h, y = np.zeros((D, N)), np.zeros_like(x)
    for t in range(x.shape[1]):
        h = np.exp(s[:, t, None] * A) * h + s[:, t, None] * b[None, :, t] * x[:, t, None]
        y[:, t] = h @ c[:, t] + skip * x[:, t]
    return y * z * ref.sigmoid(z)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def layer():
    host, dev, ad, r = _weights()
    return host, dev, ad, r, StateSpaceLayer(host["in_proj"], host["x_proj"], host["dt_proj"], host["out_proj"], **dev, length=L,
                                             slots=SLOTS)


def test_prompts_of_unequal_length_with_adapters(layer):
    host, dev, ad, r, m = layer
    u, lengths, index = r(4, C, L), [L, 1, 17, 0], [2, -1, 0, 1]
    out = m.prompt(u, _ints([3, 0, 5, 1]), _ints(lengths), adapters=ad, index=_ints(index))
    want = _reference(host, dev, ad, u, lengths, index)
    for i, n in enumerate(lengths):
        got = ref.f64(out[i, :, :n])
        assert np.abs(got - want[i, :, :n]).max(initial=0.0) <= TOL, i


def test_single_positions_continue_prompts(layer):
    host, dev, ad, r, m = layer
    u, index, slots = r(3, C, L), [1, -1, 2], _ints([4, 2, 0])
    idx, split = _ints(index), [L - 5, 3, 30]
    out = m.prompt(u, slots, _ints(split), adapters=ad, index=idx)
    want = _reference(host, dev, ad, u, [s + 5 for s in split], index)
    for k in range(5):
        now = torch.stack([u[i, :, s + k] for i, s in enumerate(split)])
        step = m.step(now, slots, adapters=ad, index=idx)
        for i, s in enumerate(split):
            assert np.abs(ref.f64(step[i]) - want[i, :, s + k]).max() <= TOL, (i, k)
    for i, s in enumerate(split):
        assert np.abs(ref.f64(out[i, :, :s]) - want[i, :, :s]).max() <= TOL


def test_prompts_resume(layer):
    host, dev, ad, r, m = layer
    u = r(2, C, 2 * L)
    slots, none = _ints([1, 5]), Adapters()
    parts = [m.prompt(u[:, :, k * L:(k + 1) * L], slots, resume=k > 0) for k in range(2)]
    want = _reference(host, dev, none, u, [2 * L] * 2, [-1, -1])
    assert np.abs(ref.f64(torch.cat(parts, 2)) - want).max() <= TOL


def test_steps_replayed_from_a_graph(layer):
    host, dev, ad, r, m = layer
    slots, idx, u = _ints([2, 3, 0, 1]), _ints([0, 1, 2, -1]), r(4, C)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.step(u, slots, adapters=ad, index=idx)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m.step(u, slots, adapters=ad, index=idx)
    for _ in range(3):
        u.copy_(r(4, C))
        before = m.conv_state.clone(), m.scan_state.clone()
        eager = m.step(u, slots, adapters=ad, index=idx).clone()
        after = m.conv_state.clone(), m.scan_state.clone()
        m.conv_state.copy_(before[0]), m.scan_state.copy_(before[1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(m.conv_state, after[0]) and torch.equal(m.scan_state, after[1])


def test_shapes_are_checked(layer):
    host, dev, ad, r, m = layer
    for bad in (r(2, C, L + 1), r(2, C + 1, L), r(2, C)):
        with pytest.raises(ValueError):
            m.prompt(bad, _ints([0, 1]))
    with pytest.raises(ValueError):
        m.step(r(2, C, 1), _ints([0, 1]))
    with pytest.raises(ValueError):
        StateSpaceLayer(host["in_proj"][:-1], host["x_proj"], host["dt_proj"], host["out_proj"], **dev, length=L, slots=SLOTS)
