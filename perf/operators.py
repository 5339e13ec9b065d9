"""What is measured of the sequence operators: the short causal convolution, the selective state space scan (both for prompts and for
single tokens) and the low-rank adapters beside a shared projection.

All tensors are channels-first, (batch, channels, positions), as everywhere in this package; parameters and scan states are float32,
activations one of the three types.  The plain forms below compute in float32 and round once at the end."""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one request's next token through a narrow layer: launch latency is all there is
        {"name": "conv_step_one", "op": "conv_step", "dtype": "f32", "B": 1, "D": 1536, "K": 4, "slots": 0},
        # a full decoding batch whose states sit in a pool of slots
        {"name": "conv_step_batch", "op": "conv_step", "dtype": "bf16", "B": 128, "D": 4096, "K": 4, "slots": 192},
        # a batch of prompts of one length
        {"name": "conv_prompt", "op": "conv", "dtype": "bf16", "B": 8, "D": 2048, "L": 2048, "K": 4, "ragged": False, "state": False},
        # prompts of unequal, odd lengths that continue from earlier chunks, in the pruned layers' own type
        {"name": "conv_ragged", "op": "conv", "dtype": "f32", "B": 5, "D": 1000, "L": 1537, "K": 3, "ragged": True, "state": True},
        {"name": "scan_step_one", "op": "scan_step", "dtype": "f32", "B": 1, "D": 1536, "N": 16, "G": 1, "slots": 0},
        {"name": "scan_step_batch", "op": "scan_step", "dtype": "bf16", "B": 128, "D": 4096, "N": 16, "G": 1, "slots": 192},
        {"name": "scan_prompt", "op": "scan", "dtype": "bf16", "B": 4, "D": 4096, "L": 2048, "N": 16, "G": 1, "ragged": False, "state": False},
        # one long document: few rows, a long axis
        {"name": "scan_long", "op": "scan", "dtype": "f32", "B": 1, "D": 1024, "L": 16384, "N": 16, "G": 1, "ragged": False, "state": False},
        # short unequal prompts (one empty, one of a single token) that continue, with two groups and a state size that is no power of two
        {"name": "scan_ragged", "op": "scan", "dtype": "f16", "B": 6, "D": 1000, "L": 777, "N": 24, "G": 2, "ragged": True, "state": True},
        # a decoding batch of many requests, each with one of 32 adapters or none
        {"name": "adapter_tokens", "op": "adapter", "dtype": "bf16", "B": 64, "C": 4096, "M": 4096, "L": 1, "R": 16, "adapters": 32},
        # prompts beside a pruned projection, in its own type
        {"name": "adapter_prompt", "op": "adapter", "dtype": "f32", "B": 8, "C": 2048, "M": 4096, "L": 1024, "R": 16, "adapters": 5},
        # short odd prompts, odd channel counts
        {"name": "adapter_odd", "op": "adapter", "dtype": "bf16", "B": 12, "C": 1001, "M": 1500, "L": 333, "R": 24, "adapters": 7},
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over the logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 0.5 / hi)))
    v = max(lo, min(hi, v))
    return v - 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(["conv", "conv_step", "scan", "scan", "scan_step", "adapter", "adapter"])
    case = {"op": op, "dtype": rng.choice(sorted(TYPES))}
    if op.endswith("_step"):
        case |= {"B": _log(rng, 1, 128), "slots": 0}
        if rng.random() < 0.5:
            case["slots"] = case["B"] + rng.randrange(64)
    else:
        case["B"] = _log(rng, 1, 12)
    if op == "adapter":
        case |= {"C": _log(rng, 64, 4096), "M": _log(rng, 64, 4096), "R": rng.choice([4, 8, 16, 24, 32, 64]), "adapters": rng.randint(1, 32)}
        if rng.random() < 0.4:
            case |= {"B": _log(rng, 1, 64), "L": 1}
        else:
            case["L"] = _log(rng, 2, max(2, min(2048, 80_000_000 // (case["B"] * (case["C"] + 2 * case["M"])))))
        return case
    groups = rng.choice([1, 1, 2, 4]) if op.startswith("scan") else 1
    case["D"] = groups * _log(rng, 64 // groups, 4096 // groups)
    if case["D"] == 3072:
        case["D"] -= groups
    if op.startswith("scan"):
        case |= {"N": rng.choice([5, 8, 16, 16, 16, 24, 32, 64]), "G": groups}
    else:
        case["K"] = rng.choice([2, 3, 4, 4])
    if op == "conv":
        case["L"] = _log(rng, 1, max(1, min(8192, 33_000_000 // (case["B"] * case["D"]))))
    elif op == "scan":
        rows = case["B"] * case["D"]
        case["L"] = _log(rng, 1, max(1, min(16384, 500_000_000 // (rows * case["N"]), 64_000_000 // (rows * TYPES[case["dtype"]].itemsize))))
    if not op.endswith("_step"):
        case |= {"ragged": rng.random() < 0.4, "state": rng.random() < 0.4}
    return case


def _lengths(case, rnd):
    """Unequal lengths, one of them the longest possible; where there are enough sequences, an empty one and one of a single position."""
    B, L = case["B"], case["L"]
    n = torch.randint(0, L + 1, (B,), generator=rnd, device="cuda", dtype=torch.int32)
    n[0] = L
    if B >= 4:
        n[1], n[2] = 0, 1
    return n


def prepare(case, seed):
    rnd = torch.Generator(device="cuda").manual_seed(seed)
    ty = TYPES[case["dtype"]]
    op, B = case["op"], case["B"]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=rnd, device="cuda") * scale

    def uniform(*shape):
        return torch.rand(shape, generator=rnd, device="cuda")

    s = {"op": op}
    if op == "adapter":
        C, M, L, R, n = (case[k] for k in ("C", "M", "L", "R", "adapters"))
        s["x"], s["base"] = normal(B, C, L).to(ty), normal(B, M, L).to(ty)
        s["down"], s["up"] = normal(n, R, C, scale=C ** -0.5).to(ty), normal(n, M, R, scale=R ** -0.5).to(ty)
        s["scale"] = 0.25 + uniform(n)
        index = torch.randint(0, n, (B,), generator=rnd, device="cuda", dtype=torch.int32)
        s["index"] = torch.where(uniform(B) < 0.1, -1, index).to(torch.int32)  # some requests have no adapter
        return s
    D = case["D"]
    step = op.endswith("_step")
    L = () if step else (case["L"],)
    # the two halves of one projection's output: strided views, as a layer has them
    xz = normal(B, 2 * D, *L).to(ty)
    s["x"] = xz[:, :D]
    pool = case["slots"] or B if step else B
    s["slots"] = None
    if step and case["slots"]:
        s["slots"] = torch.randperm(pool, generator=rnd, device="cuda")[:B].to(torch.int32)
    s["lengths"] = _lengths(case, rnd) if not step and case["ragged"] else None
    if op.startswith("conv"):
        K = case["K"]
        s["weight"], s["bias"] = normal(D, K, scale=K ** -0.5), normal(D, scale=0.1)
        if step:
            s["state"] = normal(pool, D, K - 1).to(ty)
        else:
            s["first"] = normal(B, D, K - 1).to(ty) if case["state"] else None
            s["last"] = torch.empty((B, D, K - 1), dtype=ty, device="cuda")
        return s
    N, G = case["N"], case["G"]
    s["z"] = xz[:, D:]
    # B and C: parts of another projection's output; time steps spread over 0.001 to 0.1 as such layers are set up
    bc = normal(B, 2 * G * N, *L).to(ty)
    s["B"], s["C"] = (bc[:, i * G * N:(i + 1) * G * N].unflatten(1, (G, N)) for i in range(2))
    s["dt"] = normal(B, D, *L, scale=0.5).to(ty)
    dt0 = torch.exp(math.log(1e-3) + uniform(D) * math.log(100.0))
    s["dt_bias"] = dt0 + torch.log(-torch.expm1(-dt0))
    s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(normal(D, N, scale=0.2))
    s["D"] = 1.0 + normal(D, scale=0.1)
    if step:
        s["state"] = normal(pool, D, N, scale=0.3)
    else:
        s["first"] = normal(B, D, N, scale=0.3) if case["state"] else None
        s["last"] = torch.empty((B, D, N), device="cuda")
    return s


def run(s):
    if own:
        import sparse_weight_direct_amd as sc
        if s["op"] == "conv":
            out = sc.causal_conv(s["x"], s["weight"], s["bias"], lengths=s["lengths"], initial_state=s["first"], final_state=s["last"])
            return {"out": out, "state": s["last"]}
        if s["op"] == "conv_step":
            out = sc.causal_conv_step(s["x"], s["state"], s["weight"], s["bias"], slots=s["slots"])
            return {"out": out, "state": s["state"]}
        if s["op"] == "scan":
            out = sc.selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"], lengths=s["lengths"],
                                    initial_state=s["first"], final_state=s["last"])
            return {"out": out, "state": s["last"]}
        if s["op"] == "scan_step":
            out = sc.selective_scan_step(s["x"], s["state"], s["dt"], s["A"], s["B"], s["C"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                                         slots=s["slots"])
            return {"out": out, "state": s["state"]}
        return {"out": sc.adapter_apply(s["x"], s["down"], s["up"], s["index"], scale=s["scale"], base=s["base"])}
    return {"conv": _conv, "conv_step": _conv_step, "scan": _scan, "scan_step": _scan_step, "adapter": _adapter}[s["op"]](s)


# ---- the plain forms


def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _inside(s):
    """(B, 1, L): the positions before each sequence's length."""
    x = s["x"]
    return (torch.arange(x.shape[2], device=x.device) < s["lengths"][:, None])[:, None]


def _conv(s):
    x, w = s["x"], s["weight"]
    B, D, L = x.shape
    K = w.shape[1]
    first = s["first"] if s["first"] is not None else x.new_zeros(B, D, K - 1)
    u = torch.cat([first, x], 2)
    v = (u.float().unfold(2, K, 1) * w[:, None]).sum(3) + s["bias"][:, None]
    out = _silu(v)
    if s["lengths"] is None:
        s["last"].copy_(u[:, :, L:])
    else:
        out = torch.where(_inside(s), out, 0.0)
        at = s["lengths"].long()[:, None, None] + torch.arange(K - 1, device=x.device)
        s["last"].copy_(u.gather(2, at.expand(B, D, K - 1)))
    return {"out": out.to(x.dtype), "state": s["last"]}


def _conv_step(s):
    x, w, slots = s["x"], s["weight"], s["slots"]
    old = s["state"] if slots is None else s["state"][slots.long()]
    u = torch.cat([old, x[:, :, None]], 2)
    out = _silu((u.float() * w).sum(2) + s["bias"])
    if slots is None:
        s["state"].copy_(u[:, :, 1:])
    else:
        s["state"][slots.long()] = u[:, :, 1:]
    return {"out": out.to(x.dtype), "state": s["state"]}


def _per_channel(v, D):
    """(B, G, N, ...) of the groups, for each of the D channels."""
    return v.float().repeat_interleave(D // v.shape[1], 1)


def _scan(s):
    x, A = s["x"].float(), s["A"]
    Bn, D, L = x.shape
    dt = _softplus(s["dt"].float() + s["dt_bias"][:, None])
    if s["lengths"] is not None:  # a step of no length: the state stays
        dt = torch.where(_inside(s), dt, 0.0)
    b = (dt * x)[..., None] * _per_channel(s["B"], D).transpose(2, 3)
    a = torch.exp(dt[..., None] * A[:, None])
    if s["first"] is not None:
        b[:, :, 0] += a[:, :, 0] * s["first"]
    reach = 1
    while reach < L:  # a scan by doubling: log2(L) passes over the whole tensors
        b = torch.cat([b[:, :, :reach], b[:, :, reach:] + a[:, :, reach:] * b[:, :, :-reach]], 2)
        a = torch.cat([a[:, :, :reach], a[:, :, reach:] * a[:, :, :-reach]], 2)
        reach *= 2
    s["last"].copy_(b[:, :, -1])
    y = (b * _per_channel(s["C"], D).transpose(2, 3)).sum(3) + s["D"][:, None] * x
    out = y * _silu(s["z"].float())
    if s["lengths"] is not None:
        out = torch.where(_inside(s), out, 0.0)
    return {"out": out.to(s["x"].dtype), "state": s["last"]}


def _scan_step(s):
    x, slots = s["x"].float(), s["slots"]
    D = x.shape[1]
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    old = s["state"] if slots is None else s["state"][slots.long()]
    new = torch.exp(dt[..., None] * s["A"]) * old + (dt * x)[..., None] * _per_channel(s["B"], D)
    y = (new * _per_channel(s["C"], D)).sum(2) + s["D"] * x
    if slots is None:
        s["state"].copy_(new)
    else:
        s["state"][slots.long()] = new
    return {"out": (y * _silu(s["z"].float())).to(s["x"].dtype), "state": s["state"]}


def _adapter(s):
    index = s["index"].long()
    r = index.clamp(min=0)
    low = torch.bmm(s["down"][r].float(), s["x"].float())
    delta = torch.bmm(s["up"][r].float(), low) * s["scale"][r][:, None, None]
    out = s["base"].float() + torch.where((index >= 0)[:, None, None], delta, 0.0)
    return {"out": out.to(s["x"].dtype)}


# ---- what the paths cannot do without


def work(case):
    es = TYPES[case["dtype"]].itemsize
    op, B = case["op"], case["B"]
    if op == "adapter":
        C, M, L, R = (case[k] for k in ("C", "M", "L", "R"))
        used = min(B, case["adapters"])
        return {"bytes": B * L * (C + 2 * M) * es + used * R * (C + M) * es + 4 * B, "flops": 2 * B * L * R * (C + M) + 2 * B * L * M}
    D, L = case["D"], case.get("L", 1)
    rows = B * D
    if op.startswith("conv"):
        K = case["K"]
        states = 2 if op == "conv_step" or case["state"] else 1
        return {"bytes": 2 * rows * L * es + states * rows * (K - 1) * es + 4 * D * (K + 1), "flops": rows * L * (2 * K + 4)}
    N, G = case["N"], case["G"]
    states = 2 if op == "scan_step" or case["state"] else 1
    return {"bytes": 4 * rows * L * es + 2 * B * G * N * L * es + states * 4 * rows * N + 4 * D * (N + 2), "flops": rows * L * (7 * N + 16)}


# ---- the definitions in 64 bits, one position after another


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]

    def wide(t):
        return None if t is None else t.double()

    if op == "adapter":
        out = wide(s["base"])
        for b, r in enumerate(s["index"].tolist()):
            if r >= 0:
                out[b] += float(s["scale"][r]) * (wide(s["up"][r]) @ (wide(s["down"][r]) @ wide(s["x"][b])))
        return {"out": out}
    step = op.endswith("_step")
    x = wide(s["x"])[..., None] if step else wide(s["x"])
    B, D, L = x.shape
    slots = s["slots"].tolist() if s["slots"] is not None else list(range(B))
    lengths = s["lengths"].tolist() if s["lengths"] is not None else [L] * B
    live = torch.tensor(lengths, device="cuda")
    first = wide(s["state"][slots] if step else s["first"])
    if op.startswith("conv"):
        w, K = wide(s["weight"]), s["weight"].shape[1]
        first = first if first is not None else x.new_zeros(B, D, K - 1)
        u = torch.cat([first, x], 2)
        v = wide(s["bias"])[:, None].expand(B, D, L).clone()
        for k in range(K):
            v += w[:, k, None] * u[:, :, k:k + L]
        out = v * torch.sigmoid(v)
        last = torch.stack([u[b, :, n:n + K - 1] for b, n in enumerate(lengths)])
    else:
        N = s["A"].shape[1]
        A = wide(s["A"])
        h = first if first is not None else x.new_zeros(B, D, N)
        Bm, Cm, dt, z = (wide(s[k])[..., None] if step else wide(s[k]) for k in ("B", "C", "dt", "z"))
        dt = dt + wide(s["dt_bias"])[:, None]
        dt = torch.where(dt > 30, dt, torch.log1p(torch.exp(dt)))
        share = D // Bm.shape[1]
        out = torch.empty_like(x)
        for t in range(L):
            d = dt[:, :, t, None]
            bt, ct = (m[..., t].repeat_interleave(share, 1) for m in (Bm, Cm))
            new = torch.exp(d * A) * h + d * bt * x[:, :, t, None]
            h = torch.where((live > t)[:, None, None], new, h)
            out[:, :, t] = (h * ct).sum(2)
        out = (out + wide(s["D"])[:, None] * x) * z * torch.sigmoid(z)
        last = h
    out = torch.where((torch.arange(L, device="cuda") < live[:, None])[:, None], out, 0.0)
    if not step:
        return {"out": out, "state": last}
    pool = wide(s["state"])
    pool[slots] = last
    return {"out": out[..., 0], "state": pool}
