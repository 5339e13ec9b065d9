"""The sequence operators from their definitions, in float64 on the CPU, one position after
another, each with the error that fp32 arithmetic and one final rounding may make.

Every function returns (value, bound) pairs.  U is fp32's unit roundoff.  A sum of n products has
at most (n + 1) U times the sum of their magnitudes as its error; exp2, rcp and log1p add a few U
of their value; a rounding to the output's type adds that type's unit roundoff (plus half its
smallest subnormal)."""
import numpy as np
import torch

U = 2.0 ** -24
ROUND = {torch.float32: (2.0 ** -24, 2.0 ** -150), torch.bfloat16: (2.0 ** -8, 2.0 ** -134),
         torch.float16: (2.0 ** -11, 2.0 ** -25)}


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def sigmoid(v):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-v))


def rounded(v, err, dtype):
    rel, tiny = ROUND[dtype]
    return err + rel * (np.abs(v) + err) + tiny


def _rows(B, slots, num_slots, lengths, L):
    slot = list(range(B)) if slots is None else [int(s) if 0 <= int(s) < num_slots else -1 for s in slots]
    n = [L] * B if lengths is None else [min(max(int(v), 0), L) for v in lengths]
    return slot, [0 if s < 0 else v for s, v in zip(slot, n)]


def silu_of(v, err):
    """silu and its error, given v's: the slope stays below 1.1; exp2 of a product with log2(e) is
    off by (|v| + 2) U, and 1 + e, rcp and the product by U each."""
    y = v * sigmoid(v)
    return y, 1.1 * err + (np.abs(v) + 8) * U * np.abs(y)


def causal_conv(x, weight, bias, silu, lengths, slots, initial, final):
    """(out, bound, final pool): final is the pool before the call (or None)."""
    dtype = x.dtype
    X, w = f64(x), f64(weight)
    B, D, L = X.shape
    K = w.shape[1]
    bias = np.zeros(D) if bias is None else f64(bias)
    n_slots = final.shape[0] if final is not None else initial.shape[0] if initial is not None else B
    slot, lens = _rows(B, slots, n_slots, lengths, L)
    out, bound = np.zeros((B, D, L)), np.zeros((B, D, L))
    F, P = f64(initial), f64(final)
    P = None if P is None else P.copy()
    for b in range(B):
        if slot[b] < 0:
            continue
        n = lens[b]
        u = np.concatenate([np.zeros((D, K - 1)) if F is None else F[slot[b]], X[b, :, :n]], 1)
        v, mag = np.repeat(bias[:, None], n, 1), np.repeat(np.abs(bias)[:, None], n, 1)
        for k in range(K):
            v = v + w[:, k, None] * u[:, k:k + n]
            mag = mag + np.abs(w[:, k, None] * u[:, k:k + n])
        err = (K + 2) * U * mag
        if silu:
            v, err = silu_of(v, err)
        out[b, :, :n], bound[b, :, :n] = v, rounded(v, err, dtype)
        if P is not None:
            P[slot[b]] = u[:, n:n + K - 1]
    return out, bound, P


def selective_scan(x, dt, A, Bm, Cm, D, z, dt_bias, softplus, lengths, slots, initial, final):
    """(out, bound, final pool, its bound).

    The state's error follows the recurrence itself: h = a h' + s b x gives E = a E' + what this step
    adds, which is H (the same sum over magnitudes) times U times: 4 |s A| for the rounding of the
    exponent's product and of s (softplus is off by 4 U of its value), 8 for exp2 and the products.
    Combining segments of the axis in another order at most doubles it."""
    dtype = x.dtype
    X, T, A, Bm, Cm = f64(x), f64(dt), f64(A), f64(Bm), f64(Cm)
    nb, nd, L = X.shape
    N, G = A.shape[1], Bm.shape[1]
    skip = np.zeros(nd) if D is None else f64(D)
    bias = np.zeros(nd) if dt_bias is None else f64(dt_bias)
    Z = f64(z)
    n_slots = final.shape[0] if final is not None else initial.shape[0] if initial is not None else nb
    slot, lens = _rows(nb, slots, n_slots, lengths, L)
    F, P = f64(initial), f64(final)
    P = None if P is None else P.copy()
    PB = None if P is None else np.zeros_like(P)
    out, bound = np.zeros((nb, nd, L)), np.zeros((nb, nd, L))
    share = nd // G
    for b in range(nb):
        if slot[b] < 0:
            continue
        h = np.zeros((nd, N)) if F is None else F[slot[b]].copy()
        H, E = np.abs(h), np.zeros((nd, N))
        for t in range(lens[b]):
            raw = T[b, :, t] + bias
            s = np.logaddexp(0.0, raw) if softplus else raw
            # the rounding of dt + bias moves softplus by at most its slope times that
            ds = ((U * np.abs(raw)) * sigmoid(raw) + 4 * U * s if softplus else U * np.abs(raw))[:, None]
            s = s[:, None]
            a = np.exp(s * A)
            bt, ct = (np.repeat(m[b, :, :, t], share, 0) for m in (Bm, Cm))
            xt = X[b, :, t][:, None]
            E = a * E + np.abs(A) * ds * a * H + ds * np.abs(bt * xt)
            h = a * h + s * bt * xt
            H = a * H + np.abs(s * bt * xt)
            E = E + (8 + 4 * np.abs(s * A)) * U * H
            y = (ct * h).sum(1) + skip * xt[:, 0]
            mag = (np.abs(ct) * H).sum(1) + np.abs(skip * xt[:, 0])
            err = 2 * (np.abs(ct) * E).sum(1) + (N + 3) * U * mag
            if Z is not None:
                g, ge = silu_of(Z[b, :, t], 0.0)
                y, err = y * g, np.abs(g) * err + (np.abs(y) + err) * ge + U * np.abs(y * g)
            out[b, :, t], bound[b, :, t] = y, rounded(y, err, dtype)
        if P is not None:
            P[slot[b]], PB[slot[b]] = h, rounded(h, 2 * E, torch.float32)
    return out, bound, P, PB


def adapter(x, down, up, index, scale, base):
    """(out, bound).  The intermediate (R values a position) may be held in 16 significant bits
    where the activations have fewer; fp32 activations keep it in fp32."""
    dtype = x.dtype
    X, d, u = f64(x), f64(down), f64(up)
    B, C, L = X.shape
    n, M, R = u.shape
    s = np.ones(n) if scale is None else f64(scale)
    v = np.zeros((B, M, L)) if base is None else f64(base)
    err = np.zeros((B, M, L))
    v = v.copy()
    low = 2.0 ** -16 if dtype != torch.float32 else 0.0
    for b in range(B):
        r = int(index[b])
        if 0 <= r < n:
            v[b] += s[r] * (u[r] @ (d[r] @ X[b]))
            mag = abs(s[r]) * (np.abs(u[r]) @ (np.abs(d[r]) @ np.abs(X[b])))
            err[b] = ((C + R + 8) * U + low) * mag + 2 * U * np.abs(v[b])
    return v, rounded(v, err, dtype)


def assert_within(got, want, bound, what=""):
    got = f64(got)
    assert got.shape == want.shape, (got.shape, want.shape)
    assert np.isfinite(got).all(), f"{what}: {int((~np.isfinite(got)).sum())} values not finite"
    bad = np.abs(got - want) > bound
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside their bound; first at {i}: "
                             f"{got[i]!r}, want {want[i]!r} +- {bound[i]!r}")
