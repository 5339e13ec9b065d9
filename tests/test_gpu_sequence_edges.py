"""The sequence operators at the ends of their values and arguments: infinite, extreme and absent
values in places where a result is still defined, and calls that must be refused before anything is
written.  Bounds are those of tests/sequence_ref.py unless a test states its own."""
import numpy as np
import pytest
import torch

import sequence_ref as ref
import sparse_weight_direct_amd as sc
from test_gpu_sequence import TYPES, _gen, _ints, _randn, _scan_inputs

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


# ---- states beside the last whole four


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 15, 18, 33])
def test_scan_step_infinite_input_at_any_state_size(dtype, N):
    """An infinite input with c = b and D > 0 makes every term infinite with its sign: so is the output, whatever
    N leaves of a lane's four states."""
    g = _gen(N)
    B, D = 3, 21
    x, dt = _randn(g, B, D, dtype=dtype), _randn(g, B, D, dtype=dtype)
    A, b, skip = -torch.exp(_randn(g, D, N)), _randn(g, B, 1, N, dtype=dtype), torch.ones(D, device="cuda")
    x[0, 4], x[2, 20] = INF, -INF
    state = _randn(g, B, D, N)
    out = sc.selective_scan_step(x, state, dt, A, b, b, D=skip)
    assert out[0, 4].item() == INF and out[2, 20].item() == -INF
    assert torch.equal(state[0, 4], b[0, 0].float().sign() * INF) and torch.equal(state[2, 20], b[2, 0].float().sign() * -INF)
    out[0, 4], out[2, 20] = 0.0, 0.0
    assert torch.isfinite(out).all()


# ---- steps at the ends of their type


def _scan(s, **kw):
    return sc.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"], **kw)


def _scan_ref(s, first):
    return ref.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["z"], s["dt_bias"], True, None, None, first,
                              first)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("low", ["-inf", "lowest"])
@pytest.mark.parametrize("L", [1, 2, 100, 300, 520, 1100])
def test_scan_steps_switched_off(dtype, low, L):
    """softplus of -inf, and of the type's lowest value, is 0: the position adds nothing and the state stays.
    The oracle takes -200 in their place, whose step is 1e-87."""
    g = _gen(L)
    s = _scan_inputs(g, dtype, 2, 18, L, 16, 2)
    off = torch.rand(2, 18, L, generator=g, device="cuda") < 0.4
    off[:, 3], off[0, :, 0] = True, True  # a whole channel, and the first position of a sequence
    value = -INF if low == "-inf" else torch.finfo(dtype).min
    first = _randn(g, 2, 18, 16)
    s["dt"] = torch.where(off, -200.0, s["dt"].float()).to(dtype)
    want, bound, P, PB = _scan_ref(s, first)
    s["dt"] = torch.where(off, value, s["dt"].float()).to(dtype)
    state = first.clone()
    out = _scan(s, initial_state=state, final_state=state)
    ref.assert_within(out, want, bound, "scan")
    ref.assert_within(state, P, PB, "scan state")
    assert torch.equal(state[:, 3], first[:, 3])
    if L == 1:
        state = first.clone()
        one = {k: s[k][..., 0] for k in ("x", "dt", "z", "B", "C")}
        out = sc.selective_scan_step(one["x"], state, one["dt"], s["A"], one["B"], one["C"], D=s["D"], z=one["z"],
                                     dt_bias=s["dt_bias"])
        ref.assert_within(out[:, :, None], want, bound, "scan step")
        ref.assert_within(state, P, PB, "scan step state")


def test_scan_bias_switches_channels_off():
    """-inf (and -3e38) in dt_bias: no step of the channel, ever."""
    g = _gen(31)
    for L in (1, 40, 600):
        s = _scan_inputs(g, torch.float32, 2, 24, L, 16, 1)
        first = _randn(g, 2, 24, 16)
        s["dt_bias"][5], s["dt_bias"][17] = -200.0, -200.0
        want, bound, P, PB = _scan_ref(s, first)
        s["dt_bias"][5], s["dt_bias"][17] = -INF, -3e38
        state = first.clone()
        ref.assert_within(_scan(s, initial_state=state, final_state=state), want, bound, "scan")
        ref.assert_within(state, P, PB, "scan state")
        assert torch.equal(state[:, [5, 17]], first[:, [5, 17]])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L,at", [(1, 0), (40, 25), (300, 299), (600, 310), (1100, 1099), (1100, 700)])
def test_scan_largest_steps(dtype, L, at):
    """The type's largest value is its own softplus, and exp(s A) is 0: the state is s b x, whatever came
    before.  Four fp32 roundings make it (softplus's, dt's and dt_bias's sum, s x, its product with b; softplus is off by
    4.3 units), so the state is within 8 units of 2^-24, the sum over N states within N + 12 of its
    magnitudes, and silu as in the oracle."""
    g = _gen(at)
    N = 16
    s = _scan_inputs(g, dtype, 2, 18, L, N, 1)
    most = torch.finfo(dtype).max
    tiny = 2.0 ** -125 if dtype != torch.float16 else 2.0 ** -14
    s["dt"][:, :, at] = most
    s["x"][:, :, at] = (s["x"][:, :, at].float().sign() * tiny).to(dtype)
    s["x"][:, :, at] = torch.where(s["x"][:, :, at] == 0, tiny, s["x"][:, :, at].float()).to(dtype)
    state = _randn(g, 2, 18, N)
    out = _scan(s, initial_state=state, final_state=state)
    X, T, b, c, Z = (ref.f64(s[k])[..., at] for k in ("x", "dt", "B", "C", "z"))
    h = ((T + ref.f64(s["dt_bias"])) * X)[:, :, None] * b
    y = (h * c).sum(2) + ref.f64(s["D"]) * X
    mag = np.abs(h * c).sum(2) + np.abs(ref.f64(s["D"]) * X)
    gate, ge = ref.silu_of(Z, 0.0)
    err = (N + 12) * ref.U * mag
    want, err = y * gate, np.abs(gate) * err + (np.abs(y) + err) * ge + ref.U * np.abs(y * gate)
    ref.assert_within(out[:, :, at], want, ref.rounded(want, err, dtype), "output")
    if at == L - 1:
        ref.assert_within(state, h, 8 * ref.U * np.abs(h) + 2.0 ** -126, "state")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L,at", [(1, 0), (40, 25), (600, 310), (1100, 700)])
@pytest.mark.parametrize("value", [INF, NAN])
def test_scan_steps_not_finite(dtype, L, at, value):
    """An infinite step makes the state b x infinite with that sign, a NaN makes it NaN; what came before
    and the other channels are as without it."""
    g = _gen(at)
    s = _scan_inputs(g, dtype, 2, 20, L, 1, 1, z=False)
    first = _randn(g, 2, 20, 1)
    states = [first.clone(), first.clone()]
    clean = _scan(s, initial_state=states[0], final_state=states[0])
    s["dt"][1, 7, at] = value
    out = _scan(s, initial_state=states[1], final_state=states[1])
    keep = torch.ones(2, 20, L, dtype=torch.bool, device="cuda")
    keep[1, 7, at:] = False
    assert torch.equal(out[keep], clean[keep])
    assert not torch.isfinite(out[1, 7, at:]).any() and not torch.isfinite(states[1][1, 7]).any()
    here = out[1, 7, at].item()
    if value == INF:
        assert here == INF * float(s["x"][1, 7, at].sign() * s["B"][1, 0, 0, at].sign() * s["C"][1, 0, 0, at].sign())
    else:
        assert np.isnan(here) and torch.isnan(out[1, 7, at:]).all() and torch.isnan(states[1][1, 7]).all()
    states[0][1, 7] = states[1][1, 7] = 0.0
    assert torch.equal(*states)


# ---- an infinite input where there is no skip


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L,at", [(1, 0), (40, 39), (520, 519), (600, 300)])
def test_scan_infinite_input_without_skip(dtype, L, at):
    """Without D there is no term in x itself: the output is c b s x, infinite, and not 0 times infinity."""
    g = _gen(at + 1)
    s = _scan_inputs(g, dtype, 2, 20, L, 1, 1, z=False, skip=False)
    s["x"][0, 4, at] = -INF
    want = -INF * float(s["B"][0, 0, 0, at].sign() * s["C"][0, 0, 0, at].sign())
    assert _scan(s)[0, 4, at].item() == want


# ---- adapters: values that leave a 16-bit type


def _adapter64(x, down, up, index, scale, base):
    X, d, u, s, v = ref.f64(x), ref.f64(down), ref.f64(up), ref.f64(scale), ref.f64(base).copy()
    with np.errstate(invalid="ignore"):
        for b, r in enumerate(index):
            low = s[r] * (d[r] @ X[b])
            v[b] += (u[r][:, :, None] * low[None]).sum(1)
    return v


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [1, 7, 8, 40, 260])
@pytest.mark.parametrize("R", [1, 5, 16, 24])
def test_adapter_infinite_weights(dtype, L, R):
    """An infinity in up gives one where the R values are not 0, or NaN where two of opposite sign meet; the
    rows without one are what they were.  The R values lie in 0.5 .. 1.5 times scale, C of equal sign summed."""
    g = _gen(L + R)
    B, C, M, n = 2, 12, 37, 3
    x = (torch.rand(B, C, L, generator=g, device="cuda") + 0.5).to(dtype)
    down = (torch.rand(n, R, C, generator=g, device="cuda") + 0.5).to(dtype)
    up, base = _randn(g, n, M, R, dtype=dtype), _randn(g, B, M, L, dtype=dtype)
    scale = torch.tensor([1.0, -0.75, 0.5], device="cuda")
    index = [1, 2]
    want, bound = ref.adapter(x, down, up, index, scale, base)
    for r in range(n):
        up[r, 3, 0], up[r, 20, R - 1], up[r, 36, R // 2] = INF, -INF, INF
        if R > 1:
            up[r, 11, 0], up[r, 11, 1] = INF, -INF
    exact = _adapter64(x, down, up, index, scale, base)
    out = sc.adapter_apply(x, down, up, _ints(index), scale=scale, base=base)
    got, finite = ref.f64(out), np.isfinite(exact)
    assert (~finite).any() and (got[~finite].astype(np.float32).view(np.uint32) == exact[~finite].astype(np.float32).view(np.uint32))[
        ~np.isnan(exact[~finite])].all()
    assert np.isnan(got[np.isnan(exact)]).all()
    keep = np.ones(M, bool)
    keep[[3, 11, 20, 36]] = False
    ref.assert_within(out[:, torch.tensor(keep, device="cuda")], want[:, keep], bound[:, keep], "adapter")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("R", [1, 16, 40])
def test_adapter_large_intermediate(dtype, R):
    """R values between a 16-bit type's largest and fp32's, met by weights that bring the result back."""
    g = _gen(R)
    B, C, M, n = 2, 2, 21, 1
    for L in (3, 9, 50, 300):
        big = torch.finfo(dtype).max if dtype != torch.float32 else 2.0 ** 127 * 1.9
        x = torch.zeros(B, C, L, device="cuda")
        x[:, 0], x[:, 1] = big, big * 2.0 ** -8 if dtype != torch.float16 else big  # fp16: past its range; the others: near fp32's
        down = torch.ones(n, R, C, device="cuda", dtype=dtype)
        up = (_randn(g, n, M, R) * (2.0 ** -12 if dtype == torch.float16 else 2.0 ** -100)).to(dtype)
        x, base = x.to(dtype), torch.zeros(B, M, L, device="cuda", dtype=dtype)
        want, bound = ref.adapter(x, down, up, [0, 0], None, base)
        ref.assert_within(sc.adapter_apply(x, down, up, _ints([0, 0]), base=base), want, bound, f"L {L}")


# ---- state pools without slots


def test_empty_pools_are_refused():
    """A pool of no slots holds no sequence's state; with slots that all point outside it every row is idle."""
    x, w = torch.ones(2, 8, 16, device="cuda"), torch.ones(8, 4, device="cuda")
    A, bc = -torch.ones(8, 4, device="cuda"), torch.ones(2, 1, 4, 16, device="cuda")
    cs, hs = torch.empty(0, 8, 3, device="cuda"), torch.empty(0, 8, 4, device="cuda")
    for f in (lambda: sc.causal_conv(x, w, initial_state=cs), lambda: sc.causal_conv(x, w, final_state=cs),
              lambda: sc.causal_conv_step(x[..., 0], cs, w), lambda: sc.selective_scan(x, x, A, bc, bc, initial_state=hs),
              lambda: sc.selective_scan(x, x, A, bc, bc, final_state=hs),
              lambda: sc.selective_scan_step(x[..., 0], hs, x[..., 0], A, bc[..., 0], bc[..., 0])):
        with pytest.raises((ValueError, sc.SparseConvError)):
            f()
    idle = _ints([0, 5])
    assert not sc.causal_conv(x, w, slots=idle, initial_state=cs, final_state=cs).any()
    assert not sc.selective_scan_step(x[..., 0], hs, x[..., 0], A, bc[..., 0], bc[..., 0], slots=idle).any()


# ---- gradients


def _calls(x, w, A, bc, down, up, idx, cs, hs, out):
    """Every operator, one tensor of each kind a call."""
    x1, bc1 = x[..., 0], bc[..., 0]
    return {"x": lambda: sc.causal_conv(x, w), "weight": lambda: sc.causal_conv(x, w), "state": lambda: sc.causal_conv_step(x1, cs, w),
            "out": lambda: sc.causal_conv(x, w, out=out), "A": lambda: sc.selective_scan(x, x, A, bc, bc),
            "B": lambda: sc.selective_scan(x, x, A, bc, bc), "scan state": lambda: sc.selective_scan_step(x1, hs, x1, A, bc1, bc1),
            "down": lambda: sc.adapter_apply(x, down, up, idx), "up": lambda: sc.adapter_apply(x, down, up, idx)}


@pytest.mark.parametrize("which", ["x", "weight", "state", "out", "A", "B", "scan state", "down", "up"])
def test_tensors_that_require_gradients_are_refused(which):
    """Nothing here has a gradient: a call that a graph would have to record is refused, and runs under no_grad."""
    t = dict(x=torch.ones(2, 8, 16), w=torch.ones(8, 4), A=-torch.ones(8, 4), bc=torch.ones(2, 1, 4, 16), down=torch.ones(1, 2, 8),
             up=torch.ones(1, 8, 2), idx=torch.zeros(2, dtype=torch.int32), cs=torch.zeros(2, 8, 3), hs=torch.zeros(2, 8, 4),
             out=torch.zeros(2, 8, 16))
    t = {k: v.cuda() for k, v in t.items()}
    call = _calls(**t)[which]
    want = call().clone()
    t["cs"].zero_(), t["hs"].zero_()
    key = {"weight": "w", "state": "cs", "B": "bc", "scan state": "hs"}.get(which, which)
    t[key].requires_grad_()
    before = t["cs"].detach().clone(), t["hs"].detach().clone()
    with pytest.raises(ValueError, match="gradient"):
        call()
    assert torch.equal(t["cs"], before[0]) and torch.equal(t["hs"], before[1])
    with torch.no_grad():
        assert torch.equal(call(), want)
    with torch.inference_mode():
        t["cs"].zero_(), t["hs"].zero_()
        assert torch.equal(call(), want)


def test_tensors_written_in_place_count_their_versions():
    x, w, A = torch.ones(2, 8, 16, device="cuda"), torch.ones(8, 4, device="cuda"), -torch.ones(8, 4, device="cuda")
    bc = torch.ones(2, 1, 4, 16, device="cuda")
    cs, hs, out = torch.zeros(2, 8, 3, device="cuda"), torch.zeros(2, 8, 4, device="cuda"), torch.zeros(2, 8, 16, device="cuda")
    down, up = torch.ones(1, 2, 8, device="cuda"), torch.ones(1, 8, 2, device="cuda")
    for call, written in ((lambda: sc.causal_conv_step(x[..., 0], cs, w), [cs]),
                          (lambda: sc.causal_conv(x, w, initial_state=cs, final_state=cs, out=out), [cs, out]),
                          (lambda: sc.selective_scan(x, x, A, bc, bc, final_state=hs, out=out), [hs, out]),
                          (lambda: sc.selective_scan_step(x[..., 0], hs, x[..., 0], A, bc[..., 0], bc[..., 0]), [hs]),
                          (lambda: sc.adapter_apply(x, down, up, _ints([0, 0]), base=out, out=out), [out])):
        read = [x, w, A, bc, down, up]
        before = [t._version for t in written], [t._version for t in read]
        call()
        assert all(t._version > v for t, v in zip(written, before[0]))
        assert [t._version for t in read] == before[1]


# ---- the state space layer: nothing is written by a refused call


def _layer():
    from test_gpu_ssm import SLOTS, L, _weights
    from sparse_weight_direct_amd.ssm import StateSpaceLayer
    host, dev, ad, r = _weights(3)
    m = StateSpaceLayer(host["in_proj"], host["x_proj"], host["dt_proj"], host["out_proj"], **dev, length=L, slots=SLOTS)
    m.conv_state.copy_(r(*m.conv_state.shape)), m.scan_state.copy_(r(*m.scan_state.shape))
    return m, ad, r, host, dev


def test_refused_layer_calls_leave_the_states():
    from test_gpu_ssm import C, L
    from sparse_weight_direct_amd.ssm import Adapters
    m, ad, r, _, _ = _layer()
    u, slots, good = r(2, C, L), _ints([1, 4]), _ints([0, 2])
    down, up, scale = ad.out_proj
    only = Adapters(out_proj=ad.out_proj)
    bad = [(only, None), (only, good.long()), (only, good[:1]), (only, good.cpu()), (only, [0, 1]),
           (Adapters(out_proj=(down[:, :, 1:].contiguous(), up, scale)), good), (Adapters(out_proj=(down, up[:, 1:].contiguous(), scale)), good),
           (Adapters(out_proj=(down, up[:1].contiguous(), scale)), good), (Adapters(out_proj=(down.half(), up, scale)), good),
           (Adapters(out_proj=(down, up, torch.ones(2, device="cuda"))), good), (Adapters(out_proj=(down, up.transpose(1, 2), scale)), good),
           (Adapters(out_proj=(down[0], up[0], scale)), good), (Adapters(out_proj=(down.cpu(), up, scale)), good),
           (Adapters(out_proj=(down.repeat(1, 33, 1), up.repeat(1, 1, 33), scale)), good),
           (Adapters(out_proj=(r(4 * 3 * down.shape[2] + 1)[1:].view(3, 4, -1), up, scale)), good),  # not 16-byte aligned
          
           (Adapters(in_proj=ad.out_proj), good)]
    before = m.conv_state.clone(), m.scan_state.clone()
    for adapters, index in bad:
        for call in (lambda: m.step(u[:, :, 0], slots, adapters=adapters, index=index),
                     lambda: m.prompt(u, slots, resume=True, adapters=adapters, index=index)):
            with pytest.raises((ValueError, sc.SparseConvError)):
                call()
            assert torch.equal(m.conv_state, before[0]) and torch.equal(m.scan_state, before[1])
    m.step(u[:, :, 0], slots, adapters=only, index=good)  # and the right call runs
    assert not torch.equal(m.conv_state, before[0])


def test_layer_parameters_are_checked_at_once():
    from test_gpu_ssm import SLOTS, L, D
    from sparse_weight_direct_amd.ssm import StateSpaceLayer
    _, _, _, host, dev = _layer()
    w = (host["in_proj"], host["x_proj"], host["dt_proj"], host["out_proj"])
    for name, v in (("skip", dev["skip"][1:]), ("dt_bias", dev["dt_bias"].half()), ("conv_bias", dev["conv_bias"].cpu()),
                    ("A", dev["A"].double()), ("conv_weight", dev["conv_weight"][: D // 2]), ("conv_weight", dev["conv_weight"].t())):
        with pytest.raises(ValueError):
            StateSpaceLayer(*w, **{**dev, name: v}, length=L, slots=SLOTS)


def test_layer_takes_parameters_that_require_gradients():
    from test_gpu_ssm import C, L, SLOTS
    from sparse_weight_direct_amd.ssm import StateSpaceLayer
    m, _, r, host, dev = _layer()
    same = StateSpaceLayer(host["in_proj"], host["x_proj"], host["dt_proj"], host["out_proj"], length=L, slots=SLOTS,
                           **{k: torch.nn.Parameter(v) for k, v in dev.items()})
    u, slots = r(2, C, L), _ints([1, 4])
    assert torch.equal(m.prompt(u, slots), same.prompt(u, slots)) and torch.equal(m.scan_state[slots.long()], same.scan_state[slots.long()])
