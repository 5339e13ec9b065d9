"""The attention operators from their definitions, in float64 on the CPU, each with the error that fp32 arithmetic, the
roundings that the operators document and one final rounding may make.

Every function returns (value, bound) pairs.  U is fp32's unit roundoff; a sum of n products is off by at most
(n + 1) U times the sum of their magnitudes, in any order."""
import math

import torch

from sequence_ref import ROUND, U, assert_within, f64  # noqa: F401


def wide(t):
    return None if t is None else t.detach().cpu().double()


def rounded(v, err, dtype):
    rel, tiny = ROUND[dtype]
    return err + rel * (v.abs() + err) + tiny


def visible(past, n, T, window, prefix):
    """(n, T): which of the cache's first T positions the new positions past .. past+n-1 see, pages aside."""
    i, j = past + torch.arange(n)[:, None], torch.arange(T)[None]
    seen = j <= i
    if window:
        seen &= i - j < window
    return seen | (j < prefix)


def paged_attention(q, k_pages, v_pages, table, past, lengths=None, scale=None, cap=0.0, window=0, slopes=None, prefix=None,
                    out_dtype=None):
    """(out, bound, finite): finite says where out is a finite number.  q (B, H*D, L) on any device.

    The error of a score: D + 3 roundings of the product's magnitudes; with a cap its tanh, off by 2^-22 (fp32: 4 U) of 1
    and of slope at most 1; of the bias 3 U of it; the product with log2(e), the difference from the
    maximum and exp2's own add 4 U of the largest magnitude of a score.  A weight is off by that and 4 U of itself,
    and (16-bit types) by a rounding to q's type, relative, or 2^-31 of the row's largest (fp16, whose
    weights are 2^6 at the maximum and below: 2^-25 of them).  Maxima that trail by less than 2^8 only enlarge them.  A
    relative error e_t of each weight moves sum p v / sum p by at most sum p |e_t| (|v| + |out|) / sum p."""
    dtype = q.dtype
    out_dtype = out_dtype or dtype
    Q, K, V = wide(q), wide(k_pages), wide(v_pages)
    pages, G, P, D = K.shape
    B, HD, L = Q.shape
    H = HD // D
    share = H // G
    scale = D ** -0.5 if scale is None else scale
    table = table.cpu().tolist()
    width = len(table[0]) if B else 0
    past = past.cpu().tolist()
    lengths = [L] * B if lengths is None else [min(max(int(v), 0), L) for v in lengths]
    prefix = [0] * B if prefix is None else [int(v) for v in prefix]
    slopes = None if slopes is None else wide(slopes)
    out, bound = torch.zeros(B, H, D, L, dtype=torch.float64), torch.zeros(B, H, D, L, dtype=torch.float64)
    weight_round = ROUND[dtype][0] if dtype != torch.float32 else 0.0
    Qh = Q.view(B, H, D, L)
    for b in range(B):
        n = lengths[b]
        if past[b] < 0 or past[b] > width * P or n == 0:
            continue
        T = min(past[b] + n, width * P)
        there = torch.tensor([0 <= table[b][t // P] < pages for t in range(T)], dtype=torch.bool)
        at = [max(0, table[b][t // P]) if there[t] else 0 for t in range(T)]
        kb = torch.stack([K[at[t], :, t % P] for t in range(T)], 1) if T else K.new_zeros(G, 0, D)  # (G, T, D)
        vb = torch.stack([V[at[t], :, :, t % P] for t in range(T)], 1) if T else V.new_zeros(G, 0, D)
        seen = visible(past[b], n, T, window, min(max(prefix[b], 0), T)) & there[None]
        used = seen.any(0)
        for h in range(H):
            x = Qh[b, h, :, :n].T
            k, v = kb[h // share].clone(), vb[h // share].clone()
            k[~used], v[~used] = 0.0, 0.0
            s = x @ k.T * scale
            mag = x.abs() @ k.abs().T * abs(scale)
            es = (D + 3) * U * mag
            big = mag
            if cap:
                s = cap * torch.tanh(s / cap)
                es = es + cap * (4 * U if dtype == torch.float32 else 2.0 ** -22) + 3 * U * s.abs()
            if slopes is not None:
                dist = (past[b] + torch.arange(n)[:, None] - torch.arange(T)[None]).abs() * slopes[h]
                s = s - dist
                es = es + 3 * U * dist
                big = big + dist
            s = s.masked_fill(~seen, -math.inf)
            top = s.amax(1, keepdim=True) if T else s.new_full((n, 1), -math.inf)
            p = torch.exp(s - torch.where(top > -math.inf, top, 0.0)) * seen
            total = p.sum(1, keepdim=True)
            some = total > 0
            largest = (big * seen).amax(1, keepdim=True) if T else top * 0
            # a NaN or infinite value matters where it is seen alone
            ok = torch.isfinite(v)
            vf = torch.where(ok, v, 0.0)
            o = (p @ vf) / torch.where(some, total, 1.0)
            rel = torch.where(seen, es, 0.0) + 4 * U * (largest + 1)
            num = ((p * (rel + weight_round + (T + 8) * U)) @ vf.abs()) / torch.where(some, total, 1.0)
            den = (p * (rel + weight_round + (T + 8) * U)).sum(1, keepdim=True) / torch.where(some, total, 1.0)
            e = num + den * o.abs() + 4 * U * o.abs()
            if dtype == torch.float16:
                e = e + 2.0 ** -31 * ((seen.double() @ vf.abs()) + seen.sum(1, keepdim=True) * o.abs()) / torch.where(some, total, 1.0)
            e = 1.05 * e  # second order: every relative error above is far below 0.05
            bad = (seen.double() @ (~ok).double()) > 0
            o = torch.where(some, o, 0.0).masked_fill(bad, math.nan)
            out[b, h, :, :n] = o.T
            bound[b, h, :, :n] = rounded(o, e, out_dtype).T
    finite = torch.isfinite(out)
    return out.view(B, HD, L), bound.view(B, HD, L), finite.view(B, HD, L)


def check_attention(got, want, what=""):
    out, bound, finite = want
    g = wide(got)
    assert g.shape == out.shape, (g.shape, out.shape)
    assert torch.isfinite(g[finite]).all(), f"{what}: {int((~torch.isfinite(g[finite])).sum())} values not finite"
    assert not torch.isfinite(g[~finite]).any(), f"{what}: finite where something infinite is seen"
    bad = finite & ((g - out).abs() > bound)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside their bound; first at {i}: {g[i]!r}, want {out[i]!r} +- {bound[i]!r}")


def cache_append(k, v, k_pages, v_pages, table, past, q=None, freqs=None, axes=None, positions=None, interleaved=False, lengths=None):
    """(q, its bound, k_pages, their bound, v_pages) after the call; bounds of what is not written are 0.

    An angle is off by two fp64 roundings of its turns and one fp32 rounding of the part of a turn, sine and cosine by 4 U more."""
    cdtype = k_pages.dtype
    K, V = wide(k_pages).clone(), wide(v_pages).clone()
    KB = torch.zeros_like(K)
    pages, G, P, D = K.shape
    X = {n: wide(t) for n, t in (("q", q), ("k", k), ("v", v)) if t is not None}
    B, _, L = X["k"].shape
    width = table.shape[1]
    table, past = table.cpu().tolist(), past.cpu().tolist()
    lengths = [L] * B if lengths is None else [min(max(int(n), 0), L) for n in lengths]
    pairs = 0 if freqs is None else freqs.shape[0]
    f = wide(freqs)
    ax = [0] * pairs if axes is None else axes.cpu().tolist()
    pos = None if positions is None else wide(positions)
    bound = {n: torch.zeros_like(t) for n, t in X.items()}
    for b in range(B):
        n = lengths[b] if 0 <= past[b] <= width * P else 0
        for name in ("q", "k"):
            if name not in X:
                continue
            x = X[name][b].view(-1, D, L)
            e = bound[name][b].view(-1, D, L)
            for j in range(pairs):
                if not 0 <= ax[j] < (1 if pos is None else pos.shape[1]):
                    continue
                where = past[b] + torch.arange(L).double() if pos is None else pos[b, ax[j]]
                t = where * f[j]
                m, o = (2 * j, 2 * j + 1) if interleaved else (j, j + pairs)
                a, c = x[:, m].clone(), x[:, o].clone()
                x[:, m], x[:, o] = a * t.cos() - c * t.sin(), c * t.cos() + a * t.sin()
                off = (a.abs() + c.abs()) * ((math.pi + 6) * U + t.abs() * 2.0 ** -51)
                e[:, m] = e[:, o] = off
            x[:, :, n:] = 0.0 if name == "q" else x[:, :, n:]
            e[:] = rounded(x, e, cdtype)
            e[:, :, n:] = 0.0
        for i in range(n):
            t = past[b] + i
            page = table[b][t // P] if t // P < width else -1
            if 0 <= page < pages:
                K[page, :, t % P] = X["k"][b].view(G, D, L)[:, :, i]
                KB[page, :, t % P] = bound["k"][b].view(G, D, L)[:, :, i]
                V[page, :, :, t % P] = wide(v[b].to(cdtype)).view(G, D, L)[:, :, i]
    return X.get("q"), bound.get("q"), K, KB, V


def _norm(v, err, weight, bias, center, eps):
    """norm over dim 1 of v, each value off by err, and its error: sums of C terms are off by (C + 2) U of their
    magnitudes; the root, the division and the products by U of the value each."""
    C = v.shape[1]
    m = v.mean(1, keepdim=True) if center else 0.0
    em = (err.mean(1, keepdim=True) + (C + 2) * U * v.abs().mean(1, keepdim=True)) if center else 0.0
    d = v - m
    ed = err + em + U * d.abs()
    var = (d * d).mean(1, keepdim=True) + eps
    evar = 2 * (d.abs() * ed).mean(1, keepdim=True) + (ed * ed).mean(1, keepdim=True) + (C + 4) * U * var
    by = var.sqrt().reciprocal()
    rel = 0.5 * evar / var
    rel = rel / (1 - rel).clamp(min=0.1) + 3 * U
    w = 1.0 if weight is None else wide(weight)[:, None]
    n = d * by * w
    o = n + (0.0 if bias is None else wide(bias)[:, None])
    return o, ed * by * abs(w) * (1 + rel) + n.abs() * (rel + 3 * U) + U * o.abs()


def residual_norm(x, y=None, weight=None, bias=None, post_weight=None, post_bias=None, gate=None, scale=1.0, eps=1e-6, center=False,
                  normed=True):
    """(sum, bound, out, bound)."""
    dtype = x.dtype
    r, er = wide(x), torch.zeros_like(wide(x))
    if y is not None:
        v, ev = wide(y), torch.zeros_like(r)
        if post_weight is not None:
            v, ev = _norm(v, ev, post_weight, post_bias, center, eps)
        if gate is not None:
            g = wide(gate)
            g = g if g.dim() == 3 else g[:, :, None]
            v, ev = v * g, ev * g.abs() + U * (v * g).abs()
        r = r + scale * v
        er = abs(scale) * ev + 2 * U * (scale * v).abs() + U * r.abs()
    out = eo = None
    if normed:
        out, eo = _norm(r, er, weight, bias, center, eps)
        eo = rounded(out, eo, dtype)
    return r, rounded(r, er, dtype) if y is not None else er, out, eo


def assert_near(got, want, bound, what=""):
    g = wide(got)
    assert g.shape == want.shape, (g.shape, want.shape)
    assert torch.isfinite(g).all(), f"{what}: {int((~torch.isfinite(g)).sum())} values not finite"
    bad = (g - want).abs() > bound
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside their bound; first at {i}: {g[i]!r}, want {want[i]!r} +- {bound[i]!r}")
