"""What the operators of a cache in 8 bits are measured on: the block tables and slots of a step, the store of new rows with a
scale for each block and head, those rows read back, attention over that cache, and attention over the blocks of it that a cheap
score selects.

``run`` computes each of them in elementary torch operations in 32 bits (``own`` false) or through the package's entry points
(``own`` true).  Sizes follow the package's workloads; keys have channels of unlike size as real ones do, lengths and tables are
ragged and scattered as in serving.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SMALLEST = 2.0 ** -96  # the least scale of a block: smaller values are stored as zeros


# --------------------------------------------------------------------------- cases
def blocks(name, B, N, BLOCK, lo, hi, done, cut, tight=False):
    """`done`: share of sequences that have ended, `cut`: of those that an eviction has shortened."""
    return {"name": name, "op": "blocks", "B": B, "N": N, "BLOCK": BLOCK, "lo": lo, "hi": hi, "done": done, "cut": cut, "tight": tight}


def append(name, dtype, B, KV, N, D, BLOCK, lo, hi, bounds, fused=False):
    return {"name": name, "op": "append", "dtype": dtype, "B": B, "KV": KV, "N": N, "D": D, "BLOCK": BLOCK, "lo": lo, "hi": hi,
            "bounds": bounds, "fused": fused}


def read(name, dtype, B, KV, D, BLOCK, lo, hi, part=False):
    return {"name": name, "op": "read", "dtype": dtype, "B": B, "KV": KV, "D": D, "BLOCK": BLOCK, "lo": lo, "hi": hi, "part": part}


def attend(name, dtype, B, H, KV, D, BLOCK, lo, hi, NQ=1, causal=False):
    return {"name": name, "op": "attend", "dtype": dtype, "B": B, "H": H, "KV": KV, "D": D, "BLOCK": BLOCK, "lo": lo, "hi": hi,
            "NQ": NQ, "causal": causal}


def sparse(name, dtype, B, H, KV, D, BLOCK, lo, hi, budget, first, last, NQ=1, causal=False):
    return {**attend(name, dtype, B, H, KV, D, BLOCK, lo, hi, NQ, causal), "op": "sparse", "budget": budget, "first": first, "last": last}


def listed():
    return [
        # one decode step of a ragged serving batch: a token each, some sequences done: latency is all
        blocks("blocks step", 64, 1, 32, 64, 16384, 0.05, 0.0),
        # new prompts take the places of sequences that are done, others were shortened by an eviction
        blocks("blocks prompts", 500, 2000, 16, 64, 16384, 0.3, 0.2),
        # the same decode step's rows: one a sequence, into blocks that hold earlier ones, and the summaries for a selection
        append("append step f16", "f16", 64, 4, 1, 64, 32, 64, 16384, True),
        # prompts of unlike lengths, slices of one fused projection
        append("append prompts bf16", "bf16", 4, 8, 4096, 128, 16, 1, 1024, True, fused=True),
        # a few short sequences back in 32 bits
        read("read short f32", "f32", 5, 2, 64, 8, 100, 300),
        # the past of one long sequence back in 16 bits, for a prefill over it
        read("read long bf16", "bf16", 1, 8, 128, 16, 32768, 32768),
        # the smallest call: one short sequence
        attend("attend tiny f32", "f32", 1, 4, 2, 64, 16, 100, 100),
        # decode steps: a ragged batch, one long sequence, several new rows a sequence
        attend("attend ragged f16", "f16", 64, 32, 4, 64, 32, 64, 16384),
        attend("attend long bf16", "bf16", 1, 32, 8, 128, 16, 32768, 32768),
        attend("attend rows f16", "f16", 16, 64, 8, 128, 32, 2048, 2048, NQ=4, causal=True),
        # one long sequence of which each step looks at an eighth, and a batch
        sparse("sparse long bf16", "bf16", 1, 32, 8, 128, 16, 32768, 32768, 256, 4, 16),
        sparse("sparse batch f16", "f16", 24, 32, 8, 128, 16, 1000, 12000, 64, 1, 4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["blocks", "append", "append", "read", "attend", "attend", "attend", "sparse", "sparse"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    KV, D, BLOCK = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128]), rng.choice([8, 16, 32, 64])
    H = KV * rng.choice([1, 2, 3, 4, 5, 8])
    if op == "blocks":
        B = _log(rng, 1, 1000)
        N = rng.choice([1, 1, rng.randint(2, 16), _log(rng, 17, max(18, min(4000, 1_000_000 // B)))])
        hi = _log(rng, 64, 16384)
        c = blocks("", B, N, BLOCK, max(1, hi // rng.choice([1, 4, 50])), hi, rng.choice([0.0, 0.1, 0.4]), rng.choice([0.0, 0.3]),
                   rng.random() < 0.3)
    elif op == "append":
        B = _log(rng, 1, 64)
        N = rng.choice([1, 1, rng.randint(2, 16), _log(rng, 17, max(18, min(4096, 14_000_000 // (B * KV * D))))])
        hi = _log(rng, 1, max(2, min(16384, 30_000_000 // (B * KV * D))))
        c = append("", dtype, B, KV, N, D, BLOCK, max(1, hi // rng.choice([1, 4, 50])), hi, rng.random() < 0.5, rng.random() < 0.5)
    else:
        B, NQ = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4, 7, 16])
        most = 33_000_000 if op == "read" else min(33_000_000, 1_000_000_000 * KV // (H * NQ))
        hi = _log(rng, 64, max(65, min(32768, most // (B * KV * D))))
        lo = max(1, hi // rng.choice([1, 4, 50]))
        if op == "read":
            c = read("", dtype, B, KV, D, BLOCK, lo, hi, rng.random() < 0.5)
        elif op == "attend":
            c = attend("", dtype, B, H, KV, D, BLOCK, lo, hi, NQ, rng.random() < 0.7)
        else:
            nb = -(-hi // BLOCK)
            budget = rng.randint(max(1, nb // 16), nb)
            c = sparse("", dtype, B, H, KV, D, BLOCK, lo, hi, budget, rng.randint(0, budget // 4), rng.randint(0, budget // 4), NQ,
                       rng.random() < 0.7)
    c.pop("name")
    return c


# --------------------------------------------------------------------------- work
def _mean_len(c):
    return c["lo"] if c["hi"] == c["lo"] else (c["hi"] - c["lo"]) / math.log(c["hi"] / c["lo"])


def work(c):
    B, n = c["B"], _mean_len(c)
    if c["op"] == "blocks":
        fresh = B * c["N"] / c["BLOCK"]
        return {"bytes": int(4 * (5 * B + 2 * B * c["N"] + 2 * fresh) + 8), "flops": B * c["N"]}
    e, KV, D, BLOCK = (4 if c["dtype"] == "f32" else 2), c["KV"], c["D"], c["BLOCK"]
    if c["op"] == "append":
        # new rows in, their codes out, and both back as values; each touched block's scales in and out, its summary as well
        rows = B * c["N"] * (0.75 if c["N"] > 16 else 1) * KV
        touched = B * KV * (1 + c["N"] / BLOCK)
        return {"bytes": int(2 * rows * D * (e + 1 + e) + touched * (16 + (4 * D if c["bounds"] else 0))), "flops": int(8 * rows * D)}
    if c["op"] == "read":
        rows = B * n * (0.875 if c["part"] else 1) * KV
        return {"bytes": int(2 * rows * (D * (1 + e) + 4 / BLOCK)), "flops": int(2 * rows * D)}
    rows, seen, more, ops = B * c["NQ"] * c["H"], n, 0.0, 0.0
    if c["op"] == "sparse":
        nb = n / BLOCK
        seen = min(n, c["budget"] * BLOCK)
        more = B * KV * (nb * (2 * D + 4) + min(nb, c["budget"]) * 4)
        ops = 4 * rows * D * nb
    moved = B * KV * seen * (2 * D + 8 / BLOCK) + 4 * B * seen / BLOCK + 2 * rows * D * e
    return {"bytes": int(moved + more), "flops": int(4 * rows * D * seen + ops)}


# --------------------------------------------------------------------------- inputs
def _lengths(c, g):
    u = torch.rand(c["B"], generator=g, dtype=torch.float64, device="cuda")
    n = torch.exp(math.log(c["lo"]) + (math.log(c["hi"]) - math.log(c["lo"])) * u).round().to(torch.int32)
    n[:1] = c["hi"]
    return n


def _table(c, g, width):
    per = -(-width // c["BLOCK"])
    perm = torch.randperm(c["B"] * per, generator=g, device="cuda").to(torch.int32)
    return perm.reshape(c["B"], per).contiguous()


def _channels(c, g):
    """Keys: a few channels of each head are several times the others, and lie off zero."""
    size = torch.exp(0.6 * torch.randn(c["KV"], c["D"], generator=g, device="cuda"))
    return size, 0.7 * size * torch.randn(c["KV"], c["D"], generator=g, device="cuda")


def _cache(c, g, width):
    """Codes, scales and summaries of a pool of scattered full blocks."""
    s = {"table": _table(c, g, width)}
    pool, (size, off) = s["table"].numel(), _channels(c, g)
    for x in "kv":
        r = torch.randn(pool, c["BLOCK"], c["KV"], c["D"], generator=g, device="cuda")
        r = r.mul_(size).add_(off) if x == "k" else r.mul_(0.5)
        s[x + "s"] = (r.abs().amax((1, 3)) / 127).contiguous()
        s[x + "c"] = (r / s[x + "s"][:, None, :, None]).round_().clamp_(-127, 127).to(torch.int8)
        del r
    s["bounds"] = torch.stack((s["kc"].amin(1), s["kc"].amax(1)), dim=2).contiguous()
    s["size"], s["off"] = size, off
    return s


def prepare(c, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    B = c["B"]
    if own:
        from paged_kv_cache_182_gb300 import binding as pa
    if c["op"] == "blocks":
        s = {"c": c, "lens": _lengths(c, g)}
        s["table"] = _table(c, g, c["hi"] + c["N"])
        u = torch.rand(3, B, generator=g, device="cuda")
        s["add"] = torch.ones_like(s["lens"]) if c["N"] == 1 else (u[0] * (c["N"] + 1)).to(torch.int32).clamp(max=c["N"])
        keep = torch.where(u[1] < c["cut"], s["lens"] // 2, s["lens"])
        s["keep"] = torch.where(u[2] < c["done"], torch.zeros_like(keep), keep).contiguous()
        # the pool holds what the sequences have, and what is free: more than the step needs, or about a third of that
        spare = B * (-(-c["N"] // c["BLOCK"])) // (6 if c["tight"] else 1) + 1
        pool = s["table"].numel() + spare
        s["free"] = torch.full((pool,), -1, dtype=torch.int32, device="cuda")
        s["free"][:spare] = s["table"].numel() + torch.randperm(spare, generator=g, device="cuda").to(torch.int32)
        s["count"] = torch.full((1,), spare, dtype=torch.int32, device="cuda")
        if own:
            s["plan"] = pa.BlockPlan(s["table"], s["lens"], s["free"], s["count"], BLOCK=c["BLOCK"], width=c["N"],
                                             add=s["add"], keep=s["keep"])
        return s
    KV, D, dt = c["KV"], c["D"], DTYPES[c["dtype"]]
    if c["op"] == "append":
        N = c["N"]
        s = {"c": c, "lens": _lengths(c, g), **_cache(c, g, c["hi"] + N)}
        both = torch.randn(B, N, 2 * KV, D, generator=g, device="cuda")
        both[:, :, :KV] = both[:, :, :KV] * s["size"] + s["off"]
        s["kn"], s["vn"] = (x.transpose(1, 2) for x in both.to(dt).split(KV, 2))
        if not c["fused"]:
            s["kn"], s["vn"] = s["kn"].contiguous(), s["vn"].contiguous()
        s["counts"] = torch.full((B,), N, dtype=torch.int32, device="cuda")
        if N > 16:
            s["counts"] = torch.randint(N // 2, N + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        # read back from the start of the first block that the rows went into
        s["starts"] = (s["lens"] // c["BLOCK"] * c["BLOCK"]).contiguous()
        s["back"] = (s["lens"] - s["starts"] + s["counts"]).contiguous()
        width = N + c["BLOCK"]
    elif c["op"] == "read":
        s = {"c": c, "lens": _lengths(c, g), **_cache(c, g, c["hi"])}
        s["starts"] = (s["lens"] // 8 if c["part"] else torch.zeros_like(s["lens"])).contiguous()
        s["back"] = (s["lens"] - s["starts"]).contiguous()
        width = c["hi"]
    else:
        s = {"c": c, "lens": _lengths(c, g), **_cache(c, g, c["hi"])}
        # queries that look for some of the keys: a few of the scores stand out
        q = torch.randn(B, c["H"], c["NQ"], D, generator=g, device="cuda")
        s["q"] = (q * 1.5 / s["size"].repeat_interleave(c["H"] // KV, 0)[None, :, None]).to(dt)
        s["scale"] = float(np.float32(1 / math.sqrt(D)))
    if c["op"] in ("append", "read"):
        s["ko"], s["vo"] = (torch.zeros(B, KV, width, D, dtype=dt, device="cuda") for _ in range(2))
    if own:
        cache = (s["kc"], s["vc"], s["ks"], s["vs"])
        if c["op"] in ("append", "read"):
            s["read"] = pa.Q8ReadPlan(*cache, s["table"], s["starts"], counts=s["back"], k_out=s["ko"], v_out=s["vo"])
        if c["op"] == "append":
            s["plan"] = pa.Q8AppendPlan(s["kn"], s["vn"], *cache, s["table"], s["lens"], counts=s["counts"],
                                        bounds=s["bounds"] if c["bounds"] else None)
        if c["op"] == "sparse":
            s["select"] = pa.Q8SelectPlan(s["q"], s["bounds"], s["ks"], s["table"], s["lens"], BLOCK=c["BLOCK"], budget=c["budget"],
                                          keep_first=c["first"], keep_last=c["last"])
        if c["op"] in ("attend", "sparse"):
            picked = {"selected": s["select"].selected, "counts": s["select"].counts} if c["op"] == "sparse" else {}
            s["plan"] = pa.Q8Plan(s["q"], *cache, s["table"], s["lens"], scale=s["scale"], causal=c["causal"], **picked)
    return s


# --------------------------------------------------------------------------- plain forms
def _plain_blocks(s):
    c = s["c"]
    bs, B, N, table, free = c["BLOCK"], c["B"], c["N"], s["table"], s["free"]
    maxb = table.shape[1]
    n, keep, add, count = s["lens"].long(), s["keep"].long(), s["add"].long(), s["count"].long()
    up = lambda x: (x + bs - 1) // bs  # noqa: E731
    have, need = up(n), up(keep + add)
    fits = need <= maxb
    more, less = torch.where(fits, (need - have).clamp(min=0), 0), (have - need).clamp(min=0)
    back = less.sum()
    upto = more.cumsum(0)
    granted = fits & ((more == 0) | (upto <= count + back))
    more = torch.where(granted, more, 0)
    taken = more.sum()
    i = torch.arange(maxb, device="cuda")
    # free blocks with the returned ones on top
    returned = (i >= need[:, None]) & (i < have[:, None])
    at = torch.where(returned, count + (returned.flatten().cumsum(0) - 1).view(B, maxb), free.numel())
    stack = torch.cat((free, free.new_zeros(1))).scatter(0, at.flatten(), table.flatten())[:-1]
    # taken from the top, in the order of the sequences
    fresh = (i >= have[:, None]) & (i < need[:, None]) & granted[:, None]
    order = (upto - more)[:, None] + i - have[:, None]
    table.copy_(torch.where(fresh, stack[(count + back - 1 - order).clamp(0, free.numel() - 1)], table))
    left = count + back - taken
    j = torch.arange(free.numel(), device="cuda")
    free.copy_(torch.where((j >= count) & (j < left), stack, free))
    r = torch.arange(N, device="cuda")
    token = keep[:, None] + r
    held = granted[:, None] & (r < add[:, None])
    phys = table.long().gather(1, (token // bs).clamp(max=maxb - 1))
    slots = torch.where(held, phys * bs + token % bs, -1).to(torch.int32)
    return torch.where(granted, keep + add, n).to(torch.int32), left.to(torch.int32), slots, torch.where(held, token, -1).to(torch.int32), table, free


def _codes(x, scale):
    """Nearest integers to x / scale: 64 bits, because the quotient may lie next to a half."""
    q = (x.double() / scale.double()).round().clamp(-127, 127)
    return torch.where(x.isnan(), 0.0, q)


def _scale_of(x, valid, dims):
    a = torch.where(valid & x.isfinite(), x.abs(), 0.0).amax(dims)
    return (a.double() / 127).float().clamp(min=SMALLEST)  # rounded once, as a division in 32 bits is


def _plain_append(s):
    c = s["c"]
    B, KV, N, D, bs = c["B"], c["KV"], c["N"], c["D"], c["BLOCK"]
    touched = (N + bs - 2) // bs + 1
    past, cnt = s["lens"].long()[:, None, None], s["counts"].long()[:, None, None]
    blk = past // bs + torch.arange(touched, device="cuda").view(1, -1, 1)
    token = blk * bs + torch.arange(bs, device="cuda")  # [B, touched, bs]
    fresh, old = (token >= past) & (token < past + cnt), token < past
    phys = s["table"].long().gather(1, blk[:, :, 0].clamp(max=s["table"].shape[1] - 1))
    used = fresh.any(2)
    to = phys[used]
    out = []
    for x in "kv":
        pool, scales = s[x + "c"], s[x + "s"]
        rows = s[x + "n"].transpose(1, 2).gather(1, (token - past).clamp(0, N - 1).view(B, -1, 1, 1).expand(-1, -1, KV, D))
        rows = rows.view(B, touched, bs, KV, D).float()[used]
        f, o = fresh[used][:, :, None, None], old[used][:, :, None, None]
        was = torch.where(o[:, 0, 0], scales[to], SMALLEST)
        now = torch.maximum(was, _scale_of(rows, f, (1, 3)))
        held = pool[to]
        again = _codes(held.double() * was[:, None, :, None].double(), now[:, None, :, None])
        codes = torch.where(f, _codes(rows, now[:, None, :, None]), torch.where(o, again, held.double())).to(torch.int8)
        pool[to], scales[to] = codes, now
        if x == "k" and c["bounds"]:
            there = f | o
            s["bounds"][to] = torch.stack((torch.where(there, codes, 127).amin(1), torch.where(there, codes, -127).amax(1)), 2)
        out.append(scales)
    return (*_plain_read(s), *out) + ((s["bounds"],) if c["bounds"] else ())


def _plain_read(s):
    c = s["c"]
    bs, width = c["BLOCK"], s["ko"].shape[2]
    r = torch.arange(width, device="cuda")
    token = s["starts"].long()[:, None] + r
    phys = s["table"].long().gather(1, (token // bs).clamp(max=s["table"].shape[1] - 1))
    there = (r < s["back"].long()[:, None])[:, None, :, None]
    for x in "kv":
        got = s[x + "c"][phys, token % bs].float() * s[x + "s"][phys][..., None]
        s[x + "o"].copy_(torch.where(there, got.transpose(1, 2).to(s[x + "o"].dtype), s[x + "o"]))
    return s["ko"], s["vo"]


def _attention(s, token, given):
    """Attention over the keys `token` [B, KV or 1, L] of each sequence, of which `given` are there."""
    c = s["c"]
    B, H, KV, D, NQ, bs = c["B"], c["H"], c["KV"], c["D"], c["NQ"], c["BLOCK"]
    token, given = token.expand(B, KV, -1), given.expand(B, KV, -1)
    n = s["lens"].long().view(B, 1, 1)
    phys = s["table"].long().gather(1, (token.reshape(B, -1) // bs).clamp(0, s["table"].shape[1] - 1)).view(token.shape)
    kh = torch.arange(KV, device="cuda").view(1, KV, 1)
    k, v = (s[x + "c"][phys, token % bs, kh].float() * s[x + "s"][phys, kh][..., None] for x in "kv")
    t = (s["q"].float().view(B, KV, -1, D) @ k.transpose(-1, -2)) * s["scale"]
    row = n - NQ + torch.arange(NQ, device="cuda").repeat(H // KV)  # [B, 1, rows]
    seen = (given & (token < n))[:, :, None] & ((token[:, :, None] <= row[..., None]) | (not c["causal"]))
    t = torch.where(seen, t, -math.inf)
    top = t.amax(-1, keepdim=True)
    e = torch.exp(t - torch.where(top == -math.inf, 0.0, top))
    total = e.sum(-1, keepdim=True)
    return ((e @ v) / torch.where(total == 0, 1.0, total)).view(B, H, NQ, D).to(s["q"].dtype)


def _plain_select(s):
    c = s["c"]
    B, KV, D = c["B"], c["KV"], c["D"]
    maxb = s["table"].shape[1]
    q = s["q"].float().view(B, KV, -1, D)
    qs = _scale_of(q, q.isfinite(), 3)
    qc = _codes(q, qs[..., None]).float()
    j = torch.arange(maxb, device="cuda")
    nb = ((s["lens"].long() + c["BLOCK"] - 1) // c["BLOCK"]).view(B, 1, 1)
    ends = s["bounds"][s["table"].long()].permute(3, 0, 2, 4, 1).float()  # [2, B, KV, D, blocks]
    dots = qc.clamp(max=0) @ ends[0] + qc.clamp(min=0) @ ends[1]  # whole numbers below 2^24: exact in 32 bits
    scale = qs[..., None] * s["ks"][s["table"].long()].transpose(1, 2)[:, :, None]
    score = (scale * dots).amax(2).clamp(-3.4e38, 3.4e38)
    must = (j < c["first"]) | (j >= nb - c["last"])
    rank = torch.where(j < nb, torch.where(must, math.inf, score), -math.inf)
    order = rank.sort(dim=2, descending=True, stable=True).indices  # equal scores: the lowest block first
    most = nb.clamp(max=c["budget"])
    keep = torch.zeros(B, KV, maxb, dtype=torch.bool, device="cuda").scatter(2, order, (j < most).expand(B, KV, maxb))
    place = torch.where(keep, keep.cumsum(2) - 1, c["budget"])
    picked = torch.full((B, KV, c["budget"] + 1), -1, dtype=torch.int64, device="cuda")
    return picked.scatter(2, place, j.expand(B, KV, maxb))[..., :-1], most.expand(B, KV, 1).squeeze(2)


def _plain_sparse(s):
    picked, counts = _plain_select(s)
    bs = s["c"]["BLOCK"]
    token = (picked.clamp(min=0)[..., None] * bs + torch.arange(bs, device="cuda")).flatten(2)
    out = _attention(s, token, (picked >= 0).repeat_interleave(bs, 2))
    return picked.to(torch.int32), counts.to(torch.int32), out


def _plain_attend(s):
    token = torch.arange(s["table"].shape[1] * s["c"]["BLOCK"], device="cuda").view(1, 1, -1)
    return _attention(s, token, torch.ones_like(token, dtype=torch.bool))


def run(s):
    c = s["c"]
    if own:
        got = s["plan"].run() if c["op"] in ("blocks", "append", "attend") else None
        if c["op"] == "blocks":
            return (*got, s["table"], s["free"])
        if c["op"] == "append":
            return (*s["read"].run(), s["ks"], s["vs"]) + ((s["bounds"],) if c["bounds"] else ())
        if c["op"] == "read":
            return s["read"].run()
        return got if c["op"] == "attend" else (*s["select"].run(), s["plan"].run())
    return {"blocks": _plain_blocks, "append": _plain_append, "read": _plain_read, "attend": _plain_attend, "sparse": _plain_sparse}[c["op"]](s)


# --------------------------------------------------------------------------- 64 bits
def _exact_codes(x, scale):
    """Rows in 64 bits to whole steps of `scale`, as integers."""
    return torch.clip(torch.round(torch.nan_to_num(x / scale, nan=0.0, posinf=127, neginf=-127)), -127, 127)


def _exact_scale(x):
    fine = x.abs()[torch.isfinite(x)]
    return max(float(np.float32(float(fine.max()) / 127.0)) if fine.numel() else 0.0, SMALLEST)


def _exact_append(c, s):
    bs, D = c["BLOCK"], c["D"]
    dbl, cpu = torch.float64, {k: v.cpu() for k, v in s.items() if torch.is_tensor(v)}
    scales = {x: cpu[x + "s"].to(dbl) for x in "kv"}
    out = {x: torch.zeros(s["ko"].shape, dtype=dbl) for x in "kv"}
    for b, (n, m) in enumerate(zip(cpu["lens"].tolist(), cpu["counts"].tolist())):
        first = n // bs
        for i in range(first, -(-(n + m) // bs)):
            p = int(cpu["table"][b, i])
            a, z = max(n, i * bs), min(n + m, (i + 1) * bs)
            for h in range(c["KV"]):
                for x in "kv":
                    new = cpu[x + "n"][b, h, a - n: z - n].to(dbl)
                    old = cpu[x + "c"][p, : a - i * bs, h].to(dbl) * scales[x][p, h]
                    now = max(_exact_scale(new), float(scales[x][p, h]) if len(old) else 0.0)
                    rows = torch.cat((_exact_codes(old, now), _exact_codes(new, now)))
                    scales[x][p, h] = now
                    out[x][b, h, (i - first) * bs: (i - first) * bs + len(rows)] = rows * now
    return (out["k"], out["v"], scales["k"], scales["v"]) + ((None,) if c["bounds"] else ())


def _exact_select(c, s, b, h, nb):
    """Blocks that sequence b and key head h look at: whole-number products, scores in 32 bits by their definition."""
    G = c["H"] // c["KV"]
    best = np.full(nb, -np.inf, np.float32)
    phys = s["table"][b, :nb].long()
    ends = s["bounds"][phys, h].to(torch.float64)
    for row in s["q"][b, h * G: (h + 1) * G].reshape(-1, c["D"]).to(torch.float64):
        qs = _exact_scale(row)
        w = _exact_codes(row, qs)
        dots = torch.maximum(w * ends[:, 0], w * ends[:, 1]).sum(1).cpu().numpy()
        step = (s["ks"][phys, h].to(torch.float64) * qs).cpu().numpy().astype(np.float32)
        best = np.maximum(best, (step.astype(np.float64) * dots).astype(np.float32))
    if nb <= c["budget"]:
        return np.arange(nb)
    mid = np.arange(c["first"], nb - c["last"])
    top = mid[np.lexsort((mid, -best[mid].astype(np.float64)))][: c["budget"] - c["first"] - c["last"]]
    return np.sort(np.concatenate((np.arange(c["first"]), top, np.arange(nb - c["last"], nb))))


def exact(c, seed):
    if c["op"] == "blocks":
        return None  # whole numbers
    s = prepare(c, seed)
    bs, dbl = c["BLOCK"], torch.float64
    if c["op"] == "append":
        if c["B"] * c["KV"] * (1 + c["N"] / bs) > 12000:
            return None
        return _exact_append(c, s)
    if c["op"] == "read":
        out = []
        for x in "kv":
            y = torch.zeros(s["ko"].shape, dtype=dbl, device="cuda")
            for b, (a, m) in enumerate(zip(s["starts"].tolist(), s["back"].tolist())):
                t = torch.arange(a, a + m, device="cuda")
                p = s["table"][b].long()[t // bs]
                y[b, :, :m] = (s[x + "c"][p, t % bs].to(dbl) * s[x + "s"][p].to(dbl)[..., None]).transpose(0, 1)
            out.append(y)
        return tuple(out)
    G, NQ = c["H"] // c["KV"], c["NQ"]
    out = torch.zeros(s["q"].shape, dtype=dbl, device="cuda")
    picked = torch.full((c["B"], c["KV"], c.get("budget", 1)), -1, dtype=torch.int32)
    counts = torch.zeros(c["B"], c["KV"], dtype=torch.int32)
    for b, n in enumerate(s["lens"].tolist()):
        row = n - NQ + torch.arange(NQ, device="cuda")
        for h in range(c["KV"]):
            t = torch.arange(n, device="cuda")
            if c["op"] == "sparse":
                ids = _exact_select(c, s, b, h, -(-n // bs))
                picked[b, h, : len(ids)], counts[b, h] = torch.from_numpy(ids.astype(np.int32)), len(ids)
                t = (torch.from_numpy(ids).cuda()[:, None] * bs + torch.arange(bs, device="cuda")).flatten()
                t = t[t < n]
            p = s["table"][b].long()[t // bs]
            k, v = (s[x + "c"][p, t % bs, h].to(dbl) * s[x + "s"][p, h].to(dbl)[:, None] for x in "kv")
            score = s["q"][b, h * G: (h + 1) * G].to(dbl) @ k.T * s["scale"]
            if c["causal"]:
                score = score.masked_fill(t[None, :] > row[:, None], -math.inf)
            out[b, h * G: (h + 1) * G] = torch.nan_to_num(torch.softmax(score, -1), nan=0.0) @ v
    return (picked, counts, out) if c["op"] == "sparse" else out
