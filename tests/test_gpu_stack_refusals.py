"""A stack whose scanning layers come before attending ones: a call that is refused has written no state, so that the corrected call
gives what it would have given at once.  And what a layer or a stack could never run is refused where it is made."""
import pytest
import torch

import sparse_weight_direct_amd as sc
import test_gpu_ssm as ssm
from sparse_weight_direct_amd.cache import PagePool
from sparse_weight_direct_amd.hybrid import AttentionLayer, HybridStack
from sparse_weight_direct_amd.ssm import StateSpaceLayer
from test_gpu_hybrid import D, FREQS, G, H, _ints, _layer, _randn, _weights

pytestmark = pytest.mark.gpu

C, L = ssm.C, ssm.L
REFUSED = (ValueError, TypeError, sc.SparseConvError)


def _stack(kinds, **kw):
    """Layers of those kinds: s scans, a attends, n attends without rotary positions."""
    host, dev, _, _ = ssm._weights(1)
    pool = PagePool(len(kinds), 40, G, D, page_size=16)
    layers = []
    for i, kind in enumerate(kinds):
        if kind == "s":
            layers.append(StateSpaceLayer(host["in_proj"], host["x_proj"], host["dt_proj"], host["out_proj"], **dev, length=L, slots=4))
        else:
            layers.append(_layer(pool, seed=i, layer=i)[1] if kind == "a" else AttentionLayer(*_weights(i), pool, i, length=L))
    return pool, HybridStack(layers, 1.0 + _randn(3, len(kinds) + 1, C) / 10, **kw)


def _states(stack):
    return [t.clone() for x in stack.layers if isinstance(x, StateSpaceLayer) for t in (x.conv_state, x.scan_state)]


BAD = {
    "table of another batch": lambda t: dict(table=t["table"][:1]), "table of longs": lambda t: dict(table=t["table"].long()),
    "table on the host": lambda t: dict(table=t["table"].cpu()), "no table": lambda t: dict(table=None),
    "table in columns": lambda t: dict(table=t["table"].t().contiguous().t()),
    "past of another batch": lambda t: dict(past=t["past"][:1]), "past of floats": lambda t: dict(past=t["past"].float()),
    "past with gaps": lambda t: dict(past=t["past"].repeat(2).view(2, 2)[:, 0]), "prefix of longs": lambda t: dict(prefix=t["past"].long()),
    "prefix of another batch": lambda t: dict(prefix=_ints([1])), "prefix of lists": lambda t: dict(prefix=[1, 2]),
    "positions of longs": lambda t: dict(positions=t["positions"].long()), "positions without an axis": lambda t: dict(positions=t["positions"][:, 0]),
    "positions of another length": lambda t: dict(positions=torch.cat([t["positions"]] * 2, 2)),
    "positions of no axis": lambda t: dict(positions=t["positions"][:, :0]), "positions of lists": lambda t: dict(positions=[[[1]], [[1]]]),
}


@pytest.mark.parametrize("kinds", ["sa", "asa", "ssan"])
@pytest.mark.parametrize("bad", sorted(BAD))
def test_a_refused_call_leaves_the_states(kinds, bad):
    pool, stack = _stack(kinds)
    slots, x = _ints([2, 0]), _randn(5, 2, C, L + 1)
    ids = [pool.add(), pool.add()]
    args = dict(zip(("table", "past"), pool.extend(ids, [L, L - 9])))
    lengths = _ints([L, L - 9])
    given = dict(args, positions=torch.zeros(2, 1, L, dtype=torch.int32, device="cuda"))
    other, clean = _stack(kinds)
    same = dict(zip(("table", "past"), other.extend([other.add(), other.add()], [L, L - 9])))

    def prompt(s, a):
        return s.prompt(x[:, :, :L].contiguous(), slots, lengths=lengths, **a)

    before = _states(stack)
    with pytest.raises(REFUSED):
        prompt(stack, dict(args, **BAD[bad](given)))
    assert all(torch.equal(a, b) for a, b in zip(before, _states(stack)))
    assert torch.equal(prompt(stack, args), prompt(clean, same))

    args = dict(zip(("table", "past"), pool.extend(ids, [1, 1])))
    same = dict(zip(("table", "past"), other.extend([0, 1], [1, 1])))
    given = dict(args, positions=torch.zeros(2, 1, 1, dtype=torch.int32, device="cuda"))
    before = _states(stack)
    with pytest.raises(REFUSED):
        stack.step(x[:, :, L].contiguous(), slots, **dict(args, **BAD[bad](given)))
    assert all(torch.equal(a, b) for a, b in zip(before, _states(stack)))
    now = x[:, :, L].contiguous()
    assert torch.equal(stack.step(now, slots, **args), clean.step(now, slots, **same))


def test_more_refusals_leave_the_states():
    """Positions that are not contiguous, or for a layer that turns nothing; tables wider than the operators take; lengths."""
    pool, stack = _stack("san")
    slots, x = _ints([2, 0]), _randn(5, 2, C, L)
    table, past = pool.extend([pool.add(), pool.add()], [L, L])
    right = torch.zeros(2, 1, L, dtype=torch.int32, device="cuda")
    before = _states(stack)
    for kw in (dict(positions=right), dict(lengths=_ints([1])), dict(prefix=_ints([1, 2, 3]))):
        with pytest.raises(REFUSED):
            stack.prompt(x, slots, table, past, **kw)
    with pytest.raises(REFUSED):
        stack.step(x[:, :, 0].contiguous(), slots, table[0].view(-1)[:1].expand(2, 2 ** 27), past)
    assert all(torch.equal(a, b) for a, b in zip(before, _states(stack)))
    pool, stack = _stack("sa")
    table, past = pool.extend([pool.add(), pool.add()], [L, L])
    apart = torch.zeros(2, L, 2, dtype=torch.int32, device="cuda").transpose(1, 2)[:, :1]
    before = _states(stack)
    with pytest.raises(REFUSED):
        stack.prompt(x, slots, table, past, positions=apart)
    assert all(torch.equal(a, b) for a, b in zip(before, _states(stack)))


def test_what_could_never_run_is_refused_at_once():
    pool = PagePool(1, 10, G, D, page_size=16)
    w = _weights(0)
    freqs = torch.tensor(FREQS, dtype=torch.float64, device="cuda")
    for kw in (dict(freqs=freqs.float()), dict(freqs=freqs.cpu()), dict(freqs=torch.cat([freqs, freqs])), dict(freqs=freqs[None]),
               dict(axes=torch.zeros(D // 2, dtype=torch.int32, device="cuda")), dict(freqs=freqs, axes=torch.zeros(3, dtype=torch.int32, device="cuda")),
               dict(freqs=freqs, axes=torch.zeros(D // 2, dtype=torch.int64, device="cuda")), dict(scale=float("nan")), dict(scale=1e39),
               dict(cap=-1.0), dict(cap=float("inf")), dict(scale=1e30, cap=1e-30), dict(window=-1), dict(window=0.5), dict(scale="x"),
               dict(slopes=torch.ones(H + 1, device="cuda")), dict(slopes=torch.ones(H, dtype=torch.float64, device="cuda"))):
        with pytest.raises(REFUSED):
            AttentionLayer(*w, pool, 0, length=L, **kw)
    assert (pool.pool == 0).all()
    m = AttentionLayer(*w, pool, 0, length=L, freqs=freqs)
    ones = torch.ones(2, C, device="cuda")
    for kw in (dict(scale=float("inf")), dict(scale=1e39), dict(eps=-1.0), dict(eps=float("nan")), dict(scale="x")):
        with pytest.raises(REFUSED):
            HybridStack([m], ones, **kw)
    HybridStack([m], ones, post_weights=ones[:1])
    odd = PagePool(1, 10, 1, 12, page_size=16)  # dims that no operator takes
    with pytest.raises(REFUSED):
        AttentionLayer(torch.zeros(36, C).numpy(), torch.zeros(C, 12).numpy(), odd, 0, length=L)
