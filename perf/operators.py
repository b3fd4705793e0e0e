"""What the operators around the paged cache are measured on: rotary positions (with their gradient, and fused with the store
into the cache), decode attention with modified scores and the weight that each key got, the eviction of the least attended
keys, and the gradient of attention with modified scores.

``run`` computes each of them in elementary torch operations in 32 bits (``own`` false) or through the package's entry points
(``own`` true).  Sizes follow the package's workloads; values are N(0, 1) like the workloads' own, lengths and tables ragged and
scattered as in serving.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------- cases
def rotary(name, dtype, B, H, KV, N, D, rot, far, **kw):
    c = {"name": name, "op": "rotary", "dtype": dtype, "B": B, "H": H, "KV": KV, "N": N, "D": D, "rot": rot, "far": far,
         "interleaved": False, "inverse": False, "fused": False, "scaling": "none", "append": False, "BLOCK": 16}
    return {**c, **kw}


def decode(name, dtype, B, H, KV, D, BLOCK, lo, hi, **kw):
    c = {"name": name, "op": "decode", "dtype": dtype, "B": B, "H": H, "KV": KV, "D": D, "BLOCK": BLOCK, "lo": lo, "hi": hi,
         "NQ": 1, "softcap": 0.0, "slopes": False, "window": 0, "prefix": 0, "weights": False}
    return {**c, **kw}


def evict(name, dtype, B, KV, D, BLOCK, lo, hi, budget, first, last, fresh):
    return {"name": name, "op": "evict", "dtype": dtype, "B": B, "KV": KV, "D": D, "BLOCK": BLOCK, "lo": lo, "hi": hi,
            "budget": budget, "first": first, "last": last, "fresh": fresh}


def backward(name, dtype, B, H, KV, SQ, SK, **kw):
    c = {"name": name, "op": "backward", "dtype": dtype, "B": B, "H": H, "KV": KV, "SQ": SQ, "SK": SK, "D": 128, "causal": True,
         "softcap": 0.0, "slopes": False, "window": 0, "prefix": 0}
    return {**c, **kw}


def listed():
    return [
        # a decode step of a ragged serving batch: one new token a sequence, rotated and stored in its slot
        rotary("rotary append f16", "f16", 64, 32, 4, 1, 64, 64, 16384, append=True, BLOCK=32),
        # the forward pass of a training step: queries and keys as slices of one fused projection
        rotary("rotary forward bf16", "bf16", 4, 32, 8, 2048, 128, 128, 2048, fused=True, scaling="bands"),
        # the gradient of a part-of-the-head rotation, pairs side by side, at far positions of a lengthened context
        rotary("rotary gradient f32", "f32", 3, 12, 4, 777, 80, 40, 1000000, interleaved=True, inverse=True, scaling="yarn"),
        # the smallest call: one short sequence, where latency is all
        decode("decode tiny f32", "f32", 1, 4, 2, 64, 16, 100, 100, softcap=30.0, slopes=True),
        # grouped-query decode with capped scores that also says which keys were attended to
        decode("decode capped f16", "f16", 8, 32, 8, 128, 16, 512, 4096, softcap=50.0, weights=True),
        # one long sequence with a distance bias, its weights kept for an eviction
        decode("decode long bf16", "bf16", 1, 32, 8, 128, 16, 32768, 32768, slopes=True, weights=True),
        # several new rows a sequence, a sliding window beside a prefix that stays visible
        decode("decode window f16", "f16", 16, 64, 8, 128, 32, 2048, 2048, NQ=4, softcap=30.0, window=1000, prefix=20),
        # a few short sequences a little over their budget, moved in place
        evict("evict small f32", "f32", 4, 2, 64, 16, 200, 500, 150, 4, 30, False),
        # a ragged batch, compacted in place: some sequences are under the budget
        evict("evict ragged f16", "f16", 64, 4, 64, 32, 64, 16384, 2048, 4, 256, False),
        # one long sequence, its kept tokens gathered into fresh blocks
        evict("evict long bf16", "bf16", 1, 8, 128, 16, 32768, 32768, 8192, 16, 1024, True),
        # a training step with capped scores
        backward("backward capped bf16", "bf16", 4, 32, 8, 2048, 2048, softcap=50.0),
        # odd lengths, a distance bias and a window beside a prefix
        backward("backward window f16", "f16", 2, 12, 4, 1500, 1500, slopes=True, window=500, prefix=100),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "decode", "decode", "evict", "evict", "backward"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    KV = rng.choice([1, 2, 3, 4, 8])
    H = KV * rng.choice([1, 2, 3, 4, 5, 8])
    if op == "rotary":
        D = rng.choice([64, 72, 80, 96, 128, 160, 256])
        rot = rng.choice([D, D, D // 2, 2 * rng.randint(2, D // 2)])
        B, append = _log(rng, 1, 64), rng.random() < 0.4
        N = rng.randint(1, 16) if append else _log(rng, 1, max(2, min(4096, 40_000_000 // (B * (H + KV) * D))))
        c = rotary("", dtype, B, H, KV, N, D, rot, _log(rng, 2048, 1000000), interleaved=rng.random() < 0.5,
                   inverse=not append and rng.random() < 0.5, fused=rng.random() < 0.5, append=append,
                   scaling=rng.choice(["none", "linear", "bands", "yarn"]), BLOCK=rng.choice([8, 16, 32, 64]))
    elif op == "decode":
        D, B = rng.choice([64, 128]), _log(rng, 1, 64)
        hi = _log(rng, 64, max(65, min(32768, 40_000_000 // (B * KV * D))))
        c = decode("", dtype, B, H, KV, D, rng.choice([8, 16, 32, 64]), max(1, hi // rng.choice([1, 4, 50])), hi,
                   NQ=rng.choice([1, 1, 1, 2, 4, 7, 16]), softcap=rng.choice([0.0, 20.0, 50.0]), slopes=rng.random() < 0.5,
                   window=rng.choice([0, 0, rng.randint(1, hi)]), prefix=rng.choice([0, 0, rng.randint(1, 200)]),
                   weights=rng.random() < 0.5)
    elif op == "evict":
        D, B = rng.choice([64, 128]), _log(rng, 1, 64)
        hi = _log(rng, 64, max(65, min(32768, 30_000_000 // (B * KV * D))))
        budget = rng.randint(max(1, hi // 8), hi)
        first = rng.choice([0, rng.randint(0, budget // 4)])
        c = evict("", dtype, B, KV, D, rng.choice([8, 16, 32, 64]), max(1, hi // rng.choice([1, 4, 50])), hi, budget, first,
                  rng.choice([0, rng.randint(0, budget // 4)]), rng.random() < 0.5)
    else:
        B = rng.randint(1, 3)
        S = _log(rng, 100, min(3000, int(math.sqrt(2.4e8 / (B * H)))))
        c = backward("", rng.choice(["f16", "bf16"]), B, H, KV, S, rng.choice([S, S, rng.randint(50, S)]),
                     causal=rng.random() < 0.7, softcap=rng.choice([0.0, 20.0, 50.0]), slopes=rng.random() < 0.5,
                     window=rng.choice([0, rng.randint(1, S)]), prefix=rng.choice([0, rng.randint(1, 200)]))
    c.pop("name")
    return c


# --------------------------------------------------------------------------- sizes and work
def _mean_len(c):
    return c["lo"] if c["hi"] == c["lo"] else (c["hi"] - c["lo"]) / math.log(c["hi"] / c["lo"])


def _pairs(c):
    """Visible (row, key) pairs of one head of a backward pass."""
    i, sk, w, p = np.arange(c["SQ"]), c["SK"], c["window"] or 1 << 30, min(c["prefix"], c["SK"])
    end = np.minimum(i + 1 if c["causal"] else np.minimum(i + w, sk), sk)
    return int(np.sum(p + np.maximum(0, end - np.maximum(np.maximum(i - w + 1, 0), p))))


def work(c):
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "rotary":
        rows = c["B"] * c["N"]
        moved = rows * (c["H"] + c["KV"]) * c["D"] * e * 2 + 4 * rows
        if c["append"]:  # the rotated key once more, into the cache, and the value's row there
            moved += rows * c["KV"] * c["D"] * e * 3 + 4 * rows
        return {"bytes": moved, "flops": rows * (c["H"] + c["KV"]) * c["rot"] * 3}
    if c["op"] == "decode":
        n = _mean_len(c)
        seen = min(n, c["window"] + c["prefix"] + c["NQ"]) if c["window"] else n
        rows = c["B"] * c["NQ"]
        moved = c["B"] * (seen + c["NQ"]) * 2 * c["KV"] * c["D"] * e + 2 * rows * c["H"] * c["D"] * e
        if c["weights"]:
            moved += 8 * c["B"] * n
        return {"bytes": int(moved), "flops": int(4 * rows * c["H"] * c["D"] * (seen + c["NQ"]))}
    if c["op"] == "evict":
        n, over = _mean_len(c), 1.0
        if c["hi"] == c["lo"]:
            over = float(c["hi"] > c["budget"])
        elif c["budget"] > c["lo"]:
            over = max(0.0, math.log(c["hi"] / c["budget"]) / math.log(c["hi"] / c["lo"]))
        kept = c["B"] * over * (c["budget"] - c["first"])
        return {"bytes": int(4 * c["B"] * (n + 2 * min(n, c["budget"])) + kept * 2 * c["KV"] * c["D"] * e * 2), "flops": int(c["B"] * n)}
    q, k = c["B"] * c["H"] * c["SQ"] * 128, c["B"] * c["KV"] * c["SK"] * 128
    return {"bytes": (4 * q + 4 * k) * e, "flops": 10 * 128 * c["B"] * c["H"] * _pairs(c)}


# --------------------------------------------------------------------------- rotary frequencies
SCALED = {"factor": 8.0, "original": 4096, "low": 1.0, "high": 4.0, "fast": 32.0, "slow": 1.0}


def _frequencies(rot, scaling, base=10000.0):
    """Angles per position of the rot / 2 pairs in 64 bits, and the factor on the rotated values."""
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    f, L = SCALED["factor"], SCALED["original"]
    if scaling == "linear":
        return inv / f, 1.0
    if scaling == "bands":
        turns = L * inv / (2 * math.pi)
        keep = ((turns - SCALED["low"]) / (SCALED["high"] - SCALED["low"])).clamp(0, 1)
        return inv * (keep + (1 - keep) / f), 1.0
    if scaling == "yarn":
        at = [rot * math.log(L / (2 * math.pi * b)) / (2 * math.log(base)) for b in (SCALED["fast"], SCALED["slow"])]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0, 1)
        return inv * (1 - ramp + ramp / f), 0.1 * math.log(f) + 1
    return inv, 1.0


# --------------------------------------------------------------------------- inputs
def _lengths(c, g):
    u = torch.rand(c["B"], generator=g, dtype=torch.float64, device="cuda")
    n = torch.exp(math.log(c["lo"]) + (math.log(c["hi"]) - math.log(c["lo"])) * u).round().to(torch.int32)
    n[:1] = c["hi"]
    return n


def _cache(c, g, width, extra=0):
    """Two pools of scattered blocks, a table that covers `width` tokens of each sequence, and one of `extra` more blocks."""
    bs, per = c["BLOCK"], -(-width // c["BLOCK"])
    pool = c["B"] * (per + extra)
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    r = lambda: torch.randn(pool, bs, c["KV"], c["D"], generator=g, device="cuda").to(DTYPES[c["dtype"]])  # noqa: E731
    table = perm[: c["B"] * per].reshape(c["B"], per).contiguous()
    return r(), r(), table, perm[c["B"] * per:].reshape(c["B"], extra).contiguous()


def prepare(c, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    dt, s = DTYPES[c["dtype"]], {"c": c}
    r = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(dt)  # noqa: E731
    B, KV, D = c["B"], c["KV"], c["D"]
    if c["op"] == "rotary":
        H, N = c["H"], c["N"]
        if c["fused"]:
            both = r(B, N, (H + 2 * KV) * D).view(B, N, H + 2 * KV, D).transpose(1, 2)
            s["q"], s["k"], s["v"] = both[:, :H], both[:, H:H + KV], both[:, H + KV:]
        else:
            s["q"], s["k"], s["v"] = r(B, H, N, D), r(B, KV, N, D), r(B, KV, N, D)
        start = torch.randint(0, max(1, c["far"] - N), (B, 1), generator=g, device="cuda", dtype=torch.int32)
        s["positions"] = (start + torch.arange(N, device="cuda", dtype=torch.int32)).contiguous()
        if c["append"]:
            s["kc"], s["vc"], table, _ = _cache(c, g, 256)
            at = s["positions"] % 256  # a sequence keeps its last 256 tokens' blocks here
            s["slots"] = (torch.gather(table, 1, (at // c["BLOCK"]).long()) * c["BLOCK"] + at % c["BLOCK"]).contiguous()
        inv, factor = _frequencies(c["rot"], c["scaling"])
        s["inv"], s["factor"] = inv.cuda(), factor
        if own:
            from paged_kv_cache_182_gb300 import binding as pa
            f = SCALED
            kind = {"none": None, "linear": ("linear", f["factor"]),
                    "bands": ("bands", f["factor"], f["original"], f["low"], f["high"]),
                    "yarn": ("yarn", f["factor"], f["original"], f["fast"], f["slow"])}[c["scaling"]]
            table = pa.rotary_table(c["rot"], base=10000.0, scaling=kind, device="cuda")
            if c["append"]:
                s["plan"] = pa.RotaryAppendPlan(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["kc"], s["vc"], table,
                                                interleaved=c["interleaved"])
            else:
                s["plan"] = pa.RotaryPlan(s["q"], s["k"], s["positions"], table, interleaved=c["interleaved"],
                                          inverse=c["inverse"])
        return s
    if c["op"] == "decode":
        H, NQ = c["H"], c["NQ"]
        s["lens"] = _lengths(c, g)
        s["kc"], s["vc"], s["table"], _ = _cache(c, g, c["hi"] + NQ)
        s["q"], s["kn"], s["vn"] = 2 * r(B, H, NQ, D), r(B, KV, NQ, D), r(B, KV, NQ, D)
        s["scale"] = float(np.float32(1 / math.sqrt(D)))
        _modify(c, s, B, H)
        if c["weights"]:
            width = s["table"].shape[1] * c["BLOCK"]
            s["win"] = torch.rand(B, width, generator=g, device="cuda")
            s["wout"] = torch.zeros(B, width, device="cuda")
        if own:
            from paged_kv_cache_182_gb300 import binding as pa
            s["plan"] = pa.ScoredPlan(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["kn"], s["vn"], scale=s["scale"],
                                      causal=True, softcap=c["softcap"], slopes=s["slopes"], window=c["window"],
                                      prefix=s["prefix"], key_weights=s.get("win"), key_weights_out=s.get("wout"), decay=0.9)
        return s
    if c["op"] == "evict":
        s["lens"] = _lengths(c, g)
        s["kc"], s["vc"], s["table"], new = _cache(c, g, c["hi"], -(-c["budget"] // c["BLOCK"]) if c["fresh"] else 0)
        s["dst"] = new if c["fresh"] else None
        # weights accumulated over many steps: most keys get little, some nothing at all (hidden behind a window)
        width = s["table"].shape[1] * c["BLOCK"]
        u = torch.rand(2, B, width, generator=g, device="cuda")
        s["weights"] = torch.where(u[1] < 0.1, 0.0, u[0] ** 6 * 30).contiguous()
        if own:
            from paged_kv_cache_182_gb300 import binding as pa
            s["plan"] = pa.EvictPlan(s["kc"], s["vc"], s["table"], s["lens"], s["weights"], budget=c["budget"],
                                     keep_first=c["first"], keep_last=c["last"], dst_table=s["dst"])
        return s
    H, SQ, SK = c["H"], c["SQ"], c["SK"]
    s["q"], s["k"], s["v"], s["g"] = 2 * r(B, H, SQ, D), r(B, KV, SK, D), r(B, KV, SK, D), r(B, H, SQ, D)
    s["scale"] = float(np.float32(1 / math.sqrt(D)))
    _modify(c, s, B, H)
    s["y"] = _forward(s)[0].to(dt)  # what the forward pass of the same step gave
    if own:
        from paged_kv_cache_182_gb300 import binding as pa
        s["plan"] = pa.ScoredVjpPlan(s["q"], s["k"], s["v"], s["y"], s["g"], scale=s["scale"], causal=c["causal"],
                                     softcap=c["softcap"], slopes=s["slopes"], window=c["window"], prefix=s["prefix"])
    return s


def _modify(c, s, B, H):
    s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H) if c["slopes"] else None
    s["prefix"] = (c["prefix"] - torch.arange(B, device="cuda", dtype=torch.int32) % 3).clamp(min=0).to(torch.int32) if c["prefix"] else None


# --------------------------------------------------------------------------- plain forms
def _rotate(s, x):
    c = s["c"]
    a = s["positions"].double()[:, None, :, None] * s["inv"]  # far positions: the angle needs 64 bits
    cos, sin = a.cos().float() * s["factor"], a.sin().float() * s["factor"]
    if c["inverse"]:
        sin = -sin
    x, rot = x.float(), c["rot"]
    if c["interleaved"]:
        u, v = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((u * cos - v * sin, u * sin + v * cos), dim=-1).flatten(-2)
    else:
        u, v = x[..., : rot // 2], x[..., rot // 2: rot]
        turned = torch.cat((u * cos - v * sin, u * sin + v * cos), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1).to(DTYPES[c["dtype"]])


def _scores(c, s, dots, row, key, total):
    """Modified scores: dots [B, H, rows, keys], row and key positions broadcast against [B, 1, rows, keys]."""
    t = dots * s["scale"]
    if c["softcap"]:
        t = c["softcap"] * torch.tanh(t / c["softcap"])
    far = (row - key).abs()
    if s["slopes"] is not None:
        t = t - s["slopes"].view(1, -1, 1, 1) * far
    seen = key < total
    if c["window"]:
        seen = seen & (far < c["window"])
    if c.get("causal", True):
        seen = seen & (key <= row)
    if s["prefix"] is not None:
        seen = seen | ((key < s["prefix"].view(-1, 1, 1, 1)) & (key < total))
    return torch.where(seen, t, -math.inf)


def _softmax(t):
    top = t.amax(-1, keepdim=True)
    e = torch.exp(t - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total == 0, 1.0, total)


def _forward(s):
    c = s["c"]
    G = c["H"] // c["KV"]
    k, v = (x.float().repeat_interleave(G, 1) for x in (s["k"], s["v"]))
    row = torch.arange(c["SQ"], device="cuda").view(1, 1, -1, 1)
    key = torch.arange(c["SK"], device="cuda").view(1, 1, 1, -1)
    dots = s["q"].float() @ k.transpose(-1, -2)
    p = _softmax(_scores(c, s, dots, row, key, c["SK"]))
    return p @ v, p, dots, k, v


def _plain_decode(s):
    c = s["c"]
    B, H, KV, D, NQ = c["B"], c["H"], c["KV"], c["D"], c["NQ"]
    L = s["table"].shape[1] * c["BLOCK"]
    j = torch.arange(L, device="cuda")
    slots = s["table"].long()[:, j // c["BLOCK"]] * c["BLOCK"] + j % c["BLOCK"]
    past = s["lens"].long().view(B, 1)
    # the new rows follow the cached ones: key j >= past is new row j - past
    fresh = ((j >= past) & (j < past + NQ))[:, None, :, None]
    at = (j - past).clamp(0, NQ - 1)[:, None, :, None].expand(B, KV, L, D)
    both = [torch.where(fresh, new.float().gather(2, at), pool.view(-1, KV, D)[slots].float().transpose(1, 2))
            for pool, new in ((s["kc"], s["kn"]), (s["vc"], s["vn"]))]
    dots = (s["q"].float().view(B, KV, -1, D) @ both[0].transpose(-1, -2)).view(B, H, NQ, L)
    row = (past + torch.arange(NQ, device="cuda")).view(B, 1, NQ, 1)
    p = _softmax(_scores(c, s, dots, row, j.view(1, 1, 1, -1), past.view(B, 1, 1, 1) + NQ))
    out = (p.view(B, KV, -1, L) @ both[1]).view(B, H, NQ, D).to(s["q"].dtype)
    if not c["weights"]:
        return out
    w = p.sum((1, 2)) + torch.where(j < past, 0.9 * s["win"], 0.0)
    s["wout"].copy_(torch.where(j < past + NQ, w, s["wout"]))
    return out, s["wout"]


def _plain_evict(s):
    c = s["c"]
    B, W, budget = c["B"], s["weights"].shape[1], c["budget"]
    j = torch.arange(W, device="cuda")
    n = s["lens"].long().view(B, 1)
    whole = n <= budget
    must = (j < c["first"]) | (j >= n - c["last"]) | whole
    # kept whatever they weigh, then by weight; a stable sort leaves equal weights to the lowest index
    rank = torch.where(j < n, torch.where(must, math.inf, s["weights"]), -math.inf)
    order = rank.sort(dim=1, descending=True, stable=True).indices
    keep = torch.zeros(B, W, dtype=torch.bool, device="cuda").scatter(1, order, j.expand(B, W) < torch.minimum(n, torch.full_like(n, budget)))
    new = keep.sum(1, keepdim=True)
    to = torch.where(keep, keep.cumsum(1) - 1, budget)  # a kept token's place, in order
    kept = torch.full((B, budget + 1), -1, dtype=torch.int64, device="cuda").scatter(1, to, j.expand(B, W))[:, :budget]
    held = kept >= 0
    src = kept.clamp(min=0)
    wout = torch.zeros(B, W, device="cuda")
    cols = min(budget, W)
    wout[:, :cols] = torch.where(held, s["weights"].gather(1, src), 0.0)[:, :cols]
    bs, r = c["BLOCK"], torch.arange(budget, device="cuda").expand(B, budget)
    moved = held if c["fresh"] else held & (src != r)
    dst = s["table"] if s["dst"] is None else s["dst"]
    a = (s["table"].long().gather(1, src // bs) * bs + src % bs)[moved]
    b = (dst.long().gather(1, (r // bs).clamp(max=dst.shape[1] - 1)) * bs + r % bs)[moved]
    flat = [x.view(-1, c["KV"], c["D"]) for x in (s["kc"], s["vc"])]
    flat[0][b] = flat[0][a]
    flat[1][b] = flat[1][a]
    return new.view(B).to(torch.int32), kept.to(torch.int32), wout, s["kc"], s["vc"]


def _plain_backward(s):
    c = s["c"]
    B, KV, D = c["B"], c["KV"], c["D"]
    _, p, dots, k, v = _forward(s)
    g, dt = s["g"].float(), s["q"].dtype
    delta = (s["y"].float() * g).sum(-1, keepdim=True)
    ds = p * (g @ v.transpose(-1, -2) - delta) * s["scale"]
    if c["softcap"]:
        ds = ds * (1 - torch.tanh(dots * s["scale"] / c["softcap"]) ** 2)
    fold = lambda x: x.view(B, KV, -1, c["SK"], D).sum(2)  # noqa: E731
    dq, dk, dv = ds @ k, fold(ds.transpose(-1, -2) @ s["q"].float()), fold(p.transpose(-1, -2) @ g)
    return dq.to(dt), dk.to(dt), dv.to(dt)


def run(s):
    c = s["c"]
    if own:
        got = s["plan"].run()
        return (*got, s["kc"], s["vc"]) if c["op"] == "evict" or c.get("append") else got
    if c["op"] == "rotary":
        q, k = _rotate(s, s["q"]), _rotate(s, s["k"])
        if not c["append"]:
            return q, k
        at = s["slots"].long().flatten()
        s["kc"].view(-1, c["KV"], c["D"])[at] = k.transpose(1, 2).flatten(0, 1)
        s["vc"].view(-1, c["KV"], c["D"])[at] = s["v"].transpose(1, 2).flatten(0, 1)
        return q, k, s["kc"], s["vc"]
    return {"decode": _plain_decode, "evict": _plain_evict, "backward": _plain_backward}[c["op"]](s)


# --------------------------------------------------------------------------- 64 bits
def _exact_weight(c, s, b, h, dots, row, key):
    """Softmax rows of sequence b and head h in 64 bits, and the factor that the cap leaves on a gradient."""
    t, slope = dots * s["scale"], torch.ones_like(dots)
    if c["softcap"]:
        t = c["softcap"] * torch.tanh(t / c["softcap"])
        slope = 1 - (t / c["softcap"]) ** 2
    d = (row[:, None] - key[None, :]).abs()
    if s["slopes"] is not None:
        t = t - s["slopes"][h].double() * d
    hidden = torch.zeros_like(d, dtype=torch.bool)
    if c["window"]:
        hidden |= d >= c["window"]
    if c.get("causal", True):
        hidden |= key[None, :] > row[:, None]
    if s["prefix"] is not None:
        hidden &= (key >= int(s["prefix"][b]))[None, :]
    t = t.masked_fill(hidden, -math.inf)
    p = torch.softmax(t, -1)
    return torch.nan_to_num(p, nan=0.0), slope


def exact(c, seed):
    s = prepare(c, seed)
    dbl = torch.float64
    if c["op"] == "rotary":
        half = c["rot"] // 2
        f = s["inv"].cpu().numpy()
        ang = np.remainder(s["positions"].cpu().numpy().astype(np.longdouble)[..., None] * f.astype(np.longdouble), 2 * np.pi)
        w = torch.polar(torch.full(ang.shape, s["factor"], dtype=dbl), torch.from_numpy(ang.astype(np.float64))).cuda()[:, None]
        if c["inverse"]:
            w = w.conj()
        got = []
        for x in (s["q"], s["k"]):
            y = x.to(dbl).contiguous().clone()
            part = y[..., : c["rot"]]
            part = part.unflatten(-1, (half, 2)) if c["interleaved"] else part.unflatten(-1, (2, half)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(part.contiguous()) * w)
            y[..., : c["rot"]] = z.flatten(-2) if c["interleaved"] else z.transpose(-1, -2).flatten(-2)
            got.append(y)
        if not c["append"]:
            return tuple(got)
        kc, vc = s["kc"].to(dbl).flatten(0, 1), s["vc"].to(dbl).flatten(0, 1)
        for n in range(c["N"]):
            kc[s["slots"][:, n].long()] = got[1][:, :, n]
            vc[s["slots"][:, n].long()] = s["v"][:, :, n].to(dbl)
        return (*got, kc.view(s["kc"].shape), vc.view(s["vc"].shape))
    if c["op"] == "decode":
        G, out = c["H"] // c["KV"], torch.zeros(s["q"].shape, dtype=dbl, device="cuda")
        weights = torch.zeros(s["table"].shape[0], s["table"].shape[1] * c["BLOCK"], dtype=dbl, device="cuda")
        for b, n in enumerate(s["lens"].tolist()):
            j = torch.arange(n, device="cuda")
            slots = s["table"][b].long()[j // c["BLOCK"]] * c["BLOCK"] + j % c["BLOCK"]
            row, key = n + torch.arange(c["NQ"], device="cuda"), torch.arange(n + c["NQ"], device="cuda")
            for kh in range(c["KV"]):
                k = torch.cat((s["kc"].flatten(0, 1)[slots, kh], s["kn"][b, kh])).to(dbl)
                v = torch.cat((s["vc"].flatten(0, 1)[slots, kh], s["vn"][b, kh])).to(dbl)
                for h in range(kh * G, kh * G + G):
                    p, _ = _exact_weight(c, s, b, h, s["q"][b, h].to(dbl) @ k.T, row, key)
                    out[b, h] = p @ v
                    weights[b, : n + c["NQ"]] += p.sum(0)
            if c["weights"]:
                weights[b, :n] += 0.9 * s["win"][b, :n].to(dbl)
        return (out, weights) if c["weights"] else out
    if c["op"] == "evict":
        bs, budget = c["BLOCK"], c["budget"]
        kc, vc = s["kc"].clone().flatten(0, 1), s["vc"].clone().flatten(0, 1)
        lens, table = s["lens"].tolist(), s["table"].cpu().numpy().astype(np.int64)
        dst = table if s["dst"] is None else s["dst"].cpu().numpy().astype(np.int64)
        w = s["weights"].cpu().numpy()
        kept = np.full((c["B"], budget), -1, np.int32)
        wout = np.zeros(w.shape)
        new = []
        for b, n in enumerate(lens):
            ids = np.arange(n)
            if n > budget:
                head, tail = ids[: c["first"]], ids[max(c["first"], n - c["last"]):]
                mid = ids[c["first"]: max(c["first"], n - c["last"])]
                best = mid[np.lexsort((mid, -w[b, mid]))][: budget - len(head) - len(tail)]
                ids = np.sort(np.concatenate((head, tail, best)))
            kept[b, : len(ids)] = ids
            wout[b, : len(ids)] = w[b, ids]
            new.append(len(ids))
            to = np.arange(len(ids))
            a = torch.from_numpy(table[b, ids // bs] * bs + ids % bs).cuda()
            z = torch.from_numpy(dst[b, to // bs] * bs + to % bs).cuda()
            kc[z], vc[z] = kc[a].clone(), vc[a].clone()
        ints = lambda x: torch.as_tensor(np.asarray(x, np.int32))  # noqa: E731
        return ints(new), ints(kept), torch.from_numpy(wout), kc.view(s["kc"].shape), vc.view(s["vc"].shape)
    G = c["H"] // c["KV"]
    dq = torch.zeros(s["q"].shape, dtype=dbl, device="cuda")
    dk, dv = torch.zeros(s["k"].shape, dtype=dbl, device="cuda"), torch.zeros(s["v"].shape, dtype=dbl, device="cuda")
    row, key = torch.arange(c["SQ"], device="cuda"), torch.arange(c["SK"], device="cuda")
    for b in range(c["B"]):
        for h in range(c["H"]):
            q, g, k, v = s["q"][b, h].to(dbl), s["g"][b, h].to(dbl), s["k"][b, h // G].to(dbl), s["v"][b, h // G].to(dbl)
            p, slope = _exact_weight(c, s, b, h, q @ k.T, row, key)
            d = p * (g @ v.T - (s["y"][b, h].to(dbl) * g).sum(-1, keepdim=True)) * slope * s["scale"]
            dq[b, h] = d @ k
            dk[b, h // G] += d.T @ q
            dv[b, h // G] += p.T @ g
    return dq, dk, dv
