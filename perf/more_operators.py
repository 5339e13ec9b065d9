"""What is measured of the attention operators: attention of new positions over a paged cache, rotary positions with the cache's
update, copies of pages, and the norms around a block with its residual sum.

Activations are channels-first, (batch, channels, positions), as everywhere in this package.  A cache's keys are (pages, heads,
positions, dims) and its values (pages, heads, dims, positions); a table names the pages of each sequence.  The plain forms below
compute in float32 (angles in float64) and round once at the end."""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one request's next token over a short context: launch latency is all there is
        {"name": "attend_step_one", "op": "attend", "dtype": "bf16", "B": 1, "H": 32, "G": 8, "D": 128, "L": 1, "past": 777, "P": 64,
         "ragged": False, "window": 0, "cap": 0.0, "slopes": False, "prefix": 0},
        # a full decoding batch whose contexts differ
        {"name": "attend_step_batch", "op": "attend", "dtype": "bf16", "B": 64, "H": 32, "G": 8, "D": 128, "L": 1, "past": 8191, "P": 64,
         "ragged": True, "window": 0, "cap": 0.0, "slopes": False, "prefix": 0},
        # decoding in the pruned layers' own type: every head has its keys, scores fall with the distance, only the last positions count
        {"name": "attend_step_window", "op": "attend", "dtype": "f32", "B": 24, "H": 16, "G": 16, "D": 64, "L": 1, "past": 3000, "P": 32,
         "ragged": True, "window": 1024, "cap": 0.0, "slopes": True, "prefix": 0},
        # a batch of prompts of one length
        {"name": "attend_prompt", "op": "attend", "dtype": "bf16", "B": 2, "H": 32, "G": 8, "D": 128, "L": 4096, "past": 0, "P": 64,
         "ragged": False, "window": 0, "cap": 0.0, "slopes": False, "prefix": 0},
        # the next chunk of one long document
        {"name": "attend_chunk", "op": "attend", "dtype": "bf16", "B": 1, "H": 32, "G": 8, "D": 128, "L": 512, "past": 30000, "P": 64,
         "ragged": False, "window": 0, "cap": 0.0, "slopes": False, "prefix": 0},
        # short unequal chunks (one empty, one of a single token), odd sizes, small pages, capped scores, a prefix that sees itself whole
        {"name": "attend_odd", "op": "attend", "dtype": "f16", "B": 5, "H": 6, "G": 2, "D": 80, "L": 333, "past": 1001, "P": 16,
         "ragged": True, "window": 0, "cap": 30.0, "slopes": False, "prefix": 100},
        # the next token of a decoding batch into the cache
        {"name": "append_step", "op": "append", "dtype": "bf16", "cache": "bf16", "B": 64, "H": 32, "G": 8, "D": 128, "L": 1, "past": 1000,
         "P": 64, "ragged": True, "axes": 1, "rotated": 128, "interleaved": False},
        # prompts with images in them: three coordinates a position
        {"name": "append_prompt", "op": "append", "dtype": "bf16", "cache": "bf16", "B": 2, "H": 32, "G": 8, "D": 128, "L": 4096, "past": 0,
         "P": 64, "ragged": False, "axes": 3, "rotated": 128, "interleaved": False},
        # a few requests branch: their last, half filled pages are copied in all layers
        {"name": "copy_fork", "op": "copy", "dtype": "bf16", "outer": 24, "pages": 200, "count": 6, "values": 32 * 2 * 64},
        # a pool is compacted
        {"name": "copy_compact", "op": "copy", "dtype": "bf16", "outer": 16, "pages": 512, "count": 200, "values": 32 * 8 * 128},
        # between two blocks of a decoding batch: norm after the one, sum, norm before the other
        {"name": "norm_step", "op": "norm", "dtype": "bf16", "B": 64, "C": 4096, "L": 1, "post": True, "pre": True, "gate": "none", "center": False},
        # the same for prompts, with a gate for each request's channels
        {"name": "norm_prompt", "op": "norm", "dtype": "bf16", "B": 8, "C": 2048, "L": 2048, "post": True, "pre": True, "gate": "channels",
         "center": False},
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)) - 0.5 / hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "append", "copy", "norm", "norm"])
    case = {"op": op, "dtype": rng.choice(sorted(TYPES))}
    es = TYPES[case["dtype"]].itemsize
    if op == "copy":
        case |= {"outer": _log(rng, 1, 32), "values": rng.choice([16, 32, 64]) * rng.choice([1, 2, 5, 8]) * rng.choice([64, 80, 128])}
        case["pages"] = _log(rng, 4, max(8, min(600, 250_000_000 // (case["outer"] * case["values"] * es))))
        case["count"] = _log(rng, 1, case["pages"] // 2)
        return case
    if op == "norm":
        case |= {"B": _log(rng, 1, 64), "C": _log(rng, 8, 8192), "post": rng.random() < 0.7, "pre": rng.random() < 0.8,
                 "gate": rng.choice(["none", "none", "channels", "all"]), "center": rng.random() < 0.3}
        case["L"] = 1 if rng.random() < 0.4 else _log(rng, 1, max(1, min(8192, 67_000_000 // (case["B"] * case["C"] * es))))
        return case
    G = rng.choice([1, 2, 2, 4, 8])
    case |= {"H": G * rng.choice([1, 2, 3, 4, 4, 8]), "G": G, "D": rng.choice([32, 40, 64, 64, 72, 80, 96, 128, 128, 192, 256]),
             "P": rng.choice([16, 16, 32, 64, 64, 128, 256]), "ragged": rng.random() < 0.6, "B": _log(rng, 1, 64)}
    kind = rng.choice(["step", "step", "few", "prompt", "prompt"])
    case["L"] = 1 if kind == "step" else _log(rng, 2, 16) if kind == "few" else _log(rng, 17, 2048)
    if kind == "prompt":
        case["B"] = _log(rng, 1, 8)
    if op == "attend":
        case["L"] = min(case["L"], int(math.sqrt(600_000_000 // (case["B"] * case["H"]))))
    rows = case["B"] * case["H"] * case["L"]
    if op == "append":
        room = 30_000_000 // (case["B"] * G * case["D"])  # positions of a sequence that the pools hold
        case["L"] = max(1, min(case["L"], room, 60_000_000 // (case["B"] * case["H"] * case["D"])))
        case["past"] = _log(rng, 1, max(1, min(3000, room - case["L"]))) - 1
        case |= {"cache": rng.choice(["bf16", "f16", "f32"]) if case["dtype"] == "f32" else case["dtype"], "axes": rng.choice([1, 1, 1, 2, 3]),
                 "rotated": rng.choice([case["D"], case["D"], case["D"] // 8 * 4]), "interleaved": rng.random() < 0.3}
        return case
    most = min(30_000, 400_000_000 // rows, 400_000_000 // (case["B"] * G * case["D"]))
    case["past"] = rng.choice([0, 1, 1]) * (_log(rng, 1, max(1, most - case["L"])) - 1)
    case |= {"window": rng.choice([0, 0, 0, _log(rng, 1, 4096)]), "cap": rng.choice([0.0, 0.0, 30.0, 50.0]), "slopes": rng.random() < 0.25,
             "prefix": rng.choice([0, 0, 0, _log(rng, 1, 512)])}
    return case


def _spread(case, lo, hi, rnd):
    """A whole number from lo to hi for each sequence, equally spaced, in an order of the seed's: their sum is the case's."""
    n = torch.linspace(lo, hi, case["B"], dtype=torch.float64).round().to(torch.int32) if case["B"] > 1 else torch.tensor([hi], dtype=torch.int32)
    return n.cuda()[torch.randperm(case["B"], generator=rnd, device="cuda")].contiguous()


def prepare(case, seed):
    rnd = torch.Generator(device="cuda").manual_seed(seed)
    ty = TYPES[case["dtype"]]
    op = case["op"]

    def normal(*shape, scale=1.0, dtype=None):
        return (torch.randn(shape, generator=rnd, device="cuda") * scale).to(dtype or ty)

    if op == "copy":
        s = {"op": op, "pool": normal(case["outer"], case["pages"], case["values"])}
        order = torch.randperm(case["pages"], generator=rnd, device="cuda").to(torch.int32)
        s["source"], s["target"] = order[:case["count"]].clone(), order[case["count"]:2 * case["count"]].clone()
        return s
    B, L = case["B"], case["L"]
    ends = () if L == 1 else (L,)
    if op == "norm":
        C = case["C"]
        s = {"op": op, "center": case["center"], "pre": case["pre"], "post": case["post"], "scale": 0.5}
        s["x"], s["y"] = normal(B, C, *ends, scale=2.0), normal(B, C, *ends)
        for name in ("weight", "post_weight"):
            s[name] = 1.0 + normal(C, scale=0.1, dtype=torch.float32)
        for name in ("bias", "post_bias"):
            s[name] = normal(C, scale=0.1, dtype=torch.float32) if case["center"] else None
        s["gate"] = None if case["gate"] == "none" else normal(B, C, *(ends if case["gate"] == "all" else ()))
        return s
    H, G, D, P = (case[k] for k in ("H", "G", "D", "P"))
    cache = TYPES[case.get("cache", case["dtype"])]
    s = {"op": op, "H": H}
    s["past"] = _spread(case, 0 if case["ragged"] else case["past"], case["past"], rnd)
    s["lengths"] = _spread(case, 0, L, rnd) if case["ragged"] and L > 1 else None
    # pages in any order, some of them nobody's
    width = -(-(case["past"] + L) // P)
    pages = B * width + 3
    s["table"] = torch.randperm(pages, generator=rnd, device="cuda")[:B * width].to(torch.int32).view(B, width)
    s["k_pages"], s["v_pages"] = normal(pages, G, P, D, dtype=cache), normal(pages, G, D, P, dtype=cache)
    # the parts of one projection's output: strided views, as a layer has them
    qkv = normal(B, (H + 2 * G) * D, *ends)
    s["q"] = qkv[:, :H * D]
    if op == "attend":
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H) if case["slopes"] else None
        s["prefix"] = torch.full((B,), case["prefix"], dtype=torch.int32, device="cuda") if case["prefix"] else None
        return s | {"window": case["window"], "cap": case["cap"]}
    s["k"], s["v"] = qkv[:, H * D:(H + G) * D], qkv[:, (H + G) * D:]
    pairs, axes = case["rotated"] // 2, case["axes"]
    s["interleaved"] = case["interleaved"]
    s["freqs"] = torch.pow(10000.0, -torch.arange(pairs, device="cuda", dtype=torch.float64) / pairs)
    s["axes"], s["positions"] = None, None
    if axes > 1:  # the pairs in turn; frames, rows and columns far from each other
        s["axes"] = (torch.arange(pairs, device="cuda") % axes).to(torch.int32)
        s["positions"] = torch.randint(0, 100_000, (B, axes, L), generator=rnd, device="cuda", dtype=torch.int32)
    return s


def run(s):
    if own:
        import sparse_weight_direct_amd as sc
        if s["op"] == "attend":
            f = sc.paged_attention if s["q"].dim() == 3 else sc.paged_attention_step
            more = {"lengths": s["lengths"]} if s["q"].dim() == 3 else {}
            return {"out": f(s["q"], s["k_pages"], s["v_pages"], s["table"], s["past"], window=s["window"], cap=s["cap"],
                             slopes=s["slopes"], prefix=s["prefix"], **more)}
        if s["op"] == "append":
            f = sc.cache_append if s["q"].dim() == 3 else sc.cache_append_step
            more = {"lengths": s["lengths"]} if s["q"].dim() == 3 else {}
            q = f(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["past"], q=s["q"], freqs=s["freqs"], axes=s["axes"],
                  positions=s["positions"], interleaved=s["interleaved"], **more)
            return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        if s["op"] == "copy":
            return {"pool": sc.cache_copy(s["pool"], s["source"], s["target"])}
        f = sc.residual_norm if s["x"].dim() == 3 else sc.residual_norm_step
        r, h = f(s["x"], s["y"], weight=s["weight"] if s["pre"] else None, bias=s["bias"] if s["pre"] else None,
                 post_weight=s["post_weight"] if s["post"] else None, post_bias=s["post_bias"] if s["post"] else None, gate=s["gate"],
                 scale=s["scale"], center=s["center"])
        return {"residual": r, "out": h} if s["pre"] else {"residual": r}
    return {"attend": _attend, "append": _append, "copy": _copy, "norm": _norm}[s["op"]](s)


# ---- the plain forms


def _new(s):
    """(B, L) positions of the new tokens, and which of them there are."""
    B, L = s["q"].shape[0], s["q"].shape[2] if s["q"].dim() == 3 else 1
    i = torch.arange(L, device="cuda")
    there = (i < s["lengths"][:, None]) if s["lengths"] is not None else (i < L).expand(B, L)
    return s["past"].long()[:, None] + i, there


def _attend(s):
    H = s["H"]
    _, G, P, D = s["k_pages"].shape
    q = s["q"].float().reshape(s["q"].shape[0], H, D, -1).transpose(2, 3)
    B, _, L, _ = q.shape
    at, there = _new(s)
    T = s["table"].shape[1] * P
    table = s["table"].long()
    k = s["k_pages"][table].transpose(1, 2).reshape(B, G, T, D).float()
    v = s["v_pages"][table].permute(0, 2, 1, 4, 3).reshape(B, G, T, D).float()
    score = torch.matmul(q.reshape(B, G, H // G * L, D) * D ** -0.5, k.transpose(2, 3)).view(B, H, L, T)
    if s["cap"]:
        score = s["cap"] * torch.tanh(score / s["cap"])
    key = torch.arange(T, device="cuda")
    back = at[:, :, None] - key  # (B, L, T): how far back a key is
    if s["slopes"] is not None:
        score = score - s["slopes"][:, None, None] * back.abs()[:, None]
    seen = back >= 0
    if s["window"]:
        seen = seen & (back < s["window"])
    if s["prefix"] is not None:
        seen = seen | (key < s["prefix"][:, None, None])
    end = s["past"].long() + (s["lengths"].long() if s["lengths"] is not None else L)
    seen = seen & (key < end[:, None, None]) & there[:, :, None]
    score = score.masked_fill_(~seen[:, None], -math.inf)
    top = score.amax(3, keepdim=True)
    p = torch.exp(score - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(3, keepdim=True)
    out = torch.matmul(p.view(B, G, H // G * L, T), v).view(B, H, L, D) / torch.where(total > 0, total, 1.0)
    return {"out": out.transpose(2, 3).reshape(s["q"].shape).to(s["q"].dtype)}


def _rotate(x, cos, sin, interleaved):
    """x (B, heads, D, L) with the pairs of its first 2 * pairs dims turned; cos and sin (B, pairs, L)."""
    pairs = cos.shape[1]
    turned, rest = x[:, :, :2 * pairs], x[:, :, 2 * pairs:]
    a, b = (turned[:, :, 0::2], turned[:, :, 1::2]) if interleaved else (turned[:, :, :pairs], turned[:, :, pairs:])
    cos, sin = cos[:, None], sin[:, None]
    parts = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack(parts, 3).flatten(2, 3) if interleaved else torch.cat(parts, 2)
    return torch.cat([turned, rest], 2)


def _append(s):
    _, G, P, D = s["k_pages"].shape
    B, H = s["q"].shape[0], s["H"]
    at, there = _new(s)
    where = at[:, None] if s["positions"] is None else s["positions"].long()
    which = torch.zeros(s["freqs"].shape[0], dtype=torch.long, device="cuda") if s["axes"] is None else s["axes"].long()
    angle = where[:, which].double() * s["freqs"][:, None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q, k = (_rotate(s[n].float().reshape(B, -1, D, at.shape[1]), cos, sin, s["interleaved"]) for n in ("q", "k"))
    v = s["v"].reshape(B, G, D, -1)
    q = torch.where(there[:, None, None], q, 0.0).reshape(s["q"].shape)
    page = s["table"].long().gather(1, (at // P).clamp(max=s["table"].shape[1] - 1))[there]
    slot = (at % P)[there]
    s["k_pages"][page, :, slot] = k.permute(0, 3, 1, 2)[there].to(s["k_pages"].dtype)
    s["v_pages"][page, :, :, slot] = v.permute(0, 3, 1, 2)[there].to(s["v_pages"].dtype)
    return {"q": q.to(s["k_pages"].dtype), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _copy(s):
    s["pool"][:, s["target"].long()] = s["pool"][:, s["source"].long()]
    return {"pool": s["pool"]}


def _normed(v, weight, bias, center):
    if center:
        v = v - v.mean(1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6) * weight[:, None]
    return v if bias is None else v + bias[:, None]


def _norm(s):
    B, C = s["x"].shape[:2]
    x, y = (s[n].float().view(B, C, -1) for n in ("x", "y"))
    if s["post"]:
        y = _normed(y, s["post_weight"], s["post_bias"], s["center"])
    if s["gate"] is not None:
        y = y * s["gate"].float().view(B, C, -1)
    r = x + s["scale"] * y
    out = {"residual": r.view(s["x"].shape).to(s["x"].dtype)}
    if s["pre"]:
        out["out"] = _normed(r, s["weight"], s["bias"], s["center"]).view(s["x"].shape).to(s["x"].dtype)
    return out


# ---- what the paths cannot do without


def _numbers(case, lo, hi):
    return [hi] if case["B"] == 1 else [lo + (hi - lo) * b / (case["B"] - 1) for b in range(case["B"])]


def work(case):
    es = TYPES[case["dtype"]].itemsize
    if case["op"] == "copy":
        n = case["outer"] * case["count"]
        return {"bytes": 2 * n * case["values"] * es + 8 * case["count"], "flops": 0}
    if case["op"] == "norm":
        B, C, L = case["B"], case["C"], case["L"]
        gate = {"none": 0, "channels": B * C, "all": B * C * L}[case["gate"]]
        return {"bytes": ((3 + case["pre"]) * B * C * L + gate) * es + 4 * C * (case["pre"] + case["post"]) * (1 + case["center"]),
                "flops": B * C * L * (3 + 4 * case["pre"] + 4 * case["post"])}
    B, H, G, D, L = (case[k] for k in ("B", "H", "G", "D", "L"))
    past = _numbers(case, 0 if case["ragged"] else case["past"], case["past"])
    new = _numbers(case, 0, L) if case["ragged"] and L > 1 else [L] * B
    if case["op"] == "append":
        ce = TYPES[case["cache"]].itemsize
        n = sum(new)
        return {"bytes": n * (H + 2 * G) * D * (es + ce) + 4 * n * case["axes"], "flops": n * (H + G) * case["rotated"] * 3}
    # of every pair of orders that the seed may bring the mean: keys that any query sees, and pairs of a query and a key
    keys = pairs = 0.0
    for p in past:
        for n in new if case["ragged"] else new[:1]:
            share = 1.0 / len(new) if case["ragged"] else 1.0
            T = p + n
            w = case["window"] or T + 1
            keys += share * (min(T, n + w - 1 + min(case["prefix"], max(0, p - w + 1))) if n else 0)
            pairs += share * n * min(w, p + (n + 1) / 2)
    return {"bytes": 2 * B * L * H * D * es + 2 * keys * G * D * es, "flops": 4 * pairs * H * D}


# ---- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "copy":
        new = s["pool"].clone()
        for a, b in zip(s["source"].tolist(), s["target"].tolist()):
            new[:, b] = s["pool"][:, a]
        return {"pool": new.double()}
    if s["op"] == "norm":
        return _exact_norm(s)
    return _exact_attend(s) if s["op"] == "attend" else _exact_append(s)


def _exact_norm(s):
    def over_channels(v, w, b):
        v = v.movedim(1, -1)
        if s["center"]:
            v = v - v.mean(-1, keepdim=True)
        v = v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-6) * w.double()
        return (v + b.double() if b is not None else v).movedim(-1, 1)

    y = s["y"].double()
    if s["post"]:
        y = over_channels(y, s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        g = s["gate"].double()
        y = y * (g[..., None] if g.dim() < y.dim() else g)
    r = s["x"].double() + s["scale"] * y
    return {"residual": r, "out": over_channels(r, s["weight"], s["bias"])} if s["pre"] else {"residual": r}


def _exact_attend(s):
    H = s["H"]
    _, G, P, D = s["k_pages"].shape
    q = s["q"].double().reshape(s["q"].shape[0], H, D, -1)
    B, _, _, L = q.shape
    out = torch.zeros_like(q)
    past = s["past"].tolist()
    new = s["lengths"].tolist() if s["lengths"] is not None else [L] * B
    for b in range(B):
        n, T = new[b], past[b] + new[b]
        if n == 0:
            continue
        pages = s["table"][b, :-(-T // P)].tolist()
        k = torch.cat([s["k_pages"][p].double() for p in pages], 1)[:, :T]
        v = torch.cat([s["v_pages"][p].double() for p in pages], 2)[:, :, :T]
        i, j = torch.arange(past[b], T, device="cuda")[:, None], torch.arange(T, device="cuda")
        hidden = j > i
        if s["window"]:
            hidden |= i - j >= s["window"]
        if s["prefix"] is not None:
            hidden &= j >= int(s["prefix"][b])
        for h in range(H):
            g = h // (H // G)
            a = (q[b, h, :, :n].T @ k[g].T) / math.sqrt(D)
            if s["cap"]:
                a = torch.tanh(a / s["cap"]) * s["cap"]
            if s["slopes"] is not None:
                a -= s["slopes"][h].double() * (i - j).abs()
            w = torch.softmax(a.masked_fill(hidden, -math.inf), 1)
            out[b, h, :, :n] = v[g] @ w.T
    return {"out": out.reshape(s["q"].shape)}


def _exact_append(s):
    _, G, P, D = s["k_pages"].shape
    B, H = s["q"].shape[0], s["H"]
    q, k, v = (s[n].double().reshape(B, -1, D, s["q"][0, 0].numel()).clone() for n in ("q", "k", "v"))
    L = q.shape[3]
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    past = s["past"].tolist()
    new = s["lengths"].tolist() if s["lengths"] is not None else [L] * B
    pairs = s["freqs"].shape[0]
    for b in range(B):
        n = new[b]
        q[b, :, :, n:] = 0
        for j in range(pairs):
            axis = int(s["axes"][j]) if s["axes"] is not None else 0
            t = (s["positions"][b, axis] if s["positions"] is not None else past[b] + torch.arange(L, device="cuda")).double() * s["freqs"][j]
            m, o = (2 * j, 2 * j + 1) if s["interleaved"] else (j, j + pairs)
            for x in (q, k):
                x[b, :, [m, o]] = torch.stack([x[b, :, m] * t.cos() - x[b, :, o] * t.sin(), x[b, :, m] * t.sin() + x[b, :, o] * t.cos()], 1)
        for i0 in range(past[b] // P * P, past[b] + n, P):
            lo, hi = max(i0, past[b]), min(i0 + P, past[b] + n)
            page = int(s["table"][b, i0 // P])
            k_pages[page, :, lo - i0:hi - i0] = k[b, :, :, lo - past[b]:hi - past[b]].transpose(1, 2)
            v_pages[page, :, :, lo - i0:hi - i0] = v[b, :, :, lo - past[b]:hi - past[b]]
    return {"q": q.reshape(s["q"].shape), "k_pages": k_pages, "v_pages": v_pages}
