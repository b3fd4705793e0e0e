"""Cache eviction by accumulated weight (include/pa_evict.h): refusals on the
CPU, selection and moved rows on the GPU.  Everything here is copied or
counted, so every comparison is exact."""
import ctypes

import numpy as np
import pytest
import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
A = 1 << 24


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_182_gb300 import _build

    _build.build()
    from paged_kv_cache_182_gb300 import binding

    return binding


# ------------------------------------------------------------------ reference
def kept_of(w, n, budget, first, last):
    if n <= budget:
        return list(range(n))
    ids = range(first, n - last)
    score = {j: -np.inf if np.isnan(w[j]) else float(w[j]) for j in ids}
    nan = {j for j in ids if np.isnan(w[j])}
    best = sorted(ids, key=lambda j: (j in nan, -score[j], j))[: budget - first - last]
    return list(range(first)) + sorted(best) + list(range(n - last, n))


def expect(kc, vc, table, lens, w, budget, first, last, dst):
    bs = kc.shape[1]
    rows = [x.reshape(-1, *x.shape[2:]).clone() for x in (kc, vc)]
    src = [r.clone() for r in rows]
    B = len(lens)
    kept = torch.full((B, budget), -1, dtype=torch.int32)
    wout = torch.zeros_like(w)
    new = []
    to = table if dst is None else dst
    for b, n in enumerate(lens):
        ids = kept_of(w[b].numpy(), n, budget, first, last)
        new.append(len(ids))
        kept[b, : len(ids)] = torch.tensor(ids, dtype=torch.int32)
        wout[b, : len(ids)] = w[b, ids]
        for r, j in enumerate(ids):
            s, d = int(table[b, j // bs]) * bs + j % bs, int(to[b, r // bs]) * bs + r % bs
            for x, y in zip(rows, src):
                x[d] = y[s]
    return torch.tensor(new, dtype=torch.int32), kept, wout, rows[0].view(kc.shape), rows[1].view(vc.shape)


# ------------------------------------------------------------------ CPU: refusals
def call(pa, B=2, KV=2, D=64, BLOCK=16, ptr=None, nopts=False, **o):
    vals = dict(max_blocks=8, num_blocks=32, dtype=1, budget=20, keep_first=2, keep_last=3, dst_table=None, dst_max_blocks=0,
                status=None)
    vals.update(o)
    opts = pa.EvictOpts(**vals)
    p = [(i + 1) * A for i in range(8)]
    for i, x in (ptr or {}).items():
        p[i] = x
    p = [None if x is None else ctypes.c_void_p(x) for x in p]
    return pa.LIB.pa_cache_evict(*p, B, KV, D, BLOCK, None if nopts else ctypes.byref(opts), None)


NULL, DIMS, UNSUP, ALIGN = -1, -2, -3, -4


@pytest.mark.parametrize("kw,code", [
    (dict(nopts=True), NULL), *[(dict(ptr={i: None}), NULL) for i in range(8)],
    (dict(B=-1), DIMS), (dict(KV=0), DIMS), (dict(BLOCK=0), DIMS), (dict(budget=0), DIMS), (dict(keep_first=-1), DIMS),
    (dict(keep_last=-1), DIMS), (dict(keep_first=10, keep_last=11), DIMS), (dict(max_blocks=0), DIMS), (dict(num_blocks=0), DIMS),
    (dict(max_blocks=1 << 26), DIMS), (dict(num_blocks=1 << 27), DIMS), (dict(budget=1 << 30), DIMS),
    (dict(dst_table=3 * A, dst_max_blocks=8), DIMS), (dict(dst_table=13 * A, dst_max_blocks=1), DIMS), (dict(dst_table=13 * A, dst_max_blocks=0), DIMS),
    (dict(ptr={7: 5 * A}), DIMS), (dict(ptr={6: 2 * A + 64}), DIMS), (dict(ptr={5: 4 * A}), DIMS), (dict(ptr={1: 1 * A}), DIMS),
    (dict(dtype=7), UNSUP), (dict(KV=1, D=4), UNSUP), (dict(KV=512, D=128), UNSUP), (dict(B=4097), UNSUP),
    (dict(ptr={0: A + 8}), ALIGN), (dict(ptr={4: 5 * A + 2}), ALIGN),
])
def test_refusals(pa, kw, code):
    assert call(pa, **kw) == code


def test_nothing_to_do(pa):
    assert call(pa, B=0) == 0


# ------------------------------------------------------------------ GPU
def make(seed, fmt, lens, KV, D, BLOCK, dst_tokens=0, spare=3, width_blocks=None):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    maxb = width_blocks or max(1, max(-(-n // BLOCK) for n in lens))
    nd = -(-dst_tokens // BLOCK)
    pool = B * (maxb + nd) + spare
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    table = perm[: B * maxb].view(B, maxb).contiguous()
    dst = perm[B * maxb: B * (maxb + nd)].view(B, nd).contiguous() if nd else None
    kc = torch.randn(pool, BLOCK, KV, D, generator=g).to(DT[fmt])
    vc = torch.randn(pool, BLOCK, KV, D, generator=g).to(DT[fmt])
    w = torch.rand(B, maxb * BLOCK, generator=g) ** 4
    return kc, vc, table, dst, torch.tensor(lens, dtype=torch.int32), w, g


def run(pa, kc, vc, table, dst, lens, w, budget, first, last, status=None):
    d = [x.cuda() for x in (kc, vc, table, lens, w)]
    plan = pa.EvictPlan(*d, budget=budget, keep_first=first, keep_last=last, dst_table=None if dst is None else dst.cuda(),
                        status=status)
    new, kept, wout = plan.run()
    torch.cuda.synchronize()
    assert torch.equal(d[3].cpu(), lens) and torch.equal(d[4].cpu().view(torch.int32), w.view(torch.int32))
    return new.cpu(), kept.cpu(), wout.cpu(), d[0].cpu(), d[1].cpu()


def same(got, want):
    for i, (a, b) in enumerate(zip(got, want)):
        if a.is_floating_point() and a.dtype == torch.float32:
            a, b = a.view(torch.int32), b.view(torch.int32)
        assert torch.equal(a, b), i


@pytest.mark.gpu
@pytest.mark.parametrize("fresh", [False, True])
@pytest.mark.parametrize("fmt,lens,KV,D,BLOCK,budget,first,last", [
    ("f16", [1], 1, 64, 16, 1, 0, 0),
    ("f16", [2], 1, 64, 16, 1, 0, 0),
    ("f32", [0, 1, 17, 40, 33], 2, 64, 16, 16, 1, 2),
    ("bf16", [300, 299, 1, 150, 151], 8, 128, 16, 150, 4, 30),
    ("f16", [5000, 4097, 100, 2500], 4, 64, 32, 1000, 7, 0),
    ("f16", [700] * 9, 1, 64, 8, 699, 0, 0),
    ("bf16", [20000, 16385], 2, 128, 64, 3000, 0, 500),
    ("f32", [513, 1024], 3, 8, 5, 200, 0, 199),
    ("f16", [900], 2, 64, 16, 40, 20, 20),   # nothing of the middle
    ("f16", [64, 50], 128, 128, 16, 30, 0, 0),  # rows of 32 KB
    ("bf16", [40, 3, 64], 2, 64, 16, 5000, 10, 20),  # a budget beyond the table
])
def test_selects_and_moves(pa, fmt, lens, KV, D, BLOCK, budget, first, last, fresh):
    kc, vc, table, dst, ln, w, _ = make(len(lens) + budget, fmt, lens, KV, D, BLOCK, budget if fresh else 0)
    want = expect(kc, vc, table, lens, w, budget, first, last, dst)
    same(run(pa, kc, vc, table, dst, ln, w, budget, first, last), want)


@pytest.mark.gpu
@pytest.mark.parametrize("lens,KV,D,BLOCK,budget,first,last", [
    ([9000], 2, 128, 32, 7100, 0, 900),          # 32-byte slices, many runs of 512 rows
    ([4000, 3900], 8, 128, 16, 3000, 5, 0),      # 64-byte ones or narrower
    ([5000] * 10, 8, 128, 16, 1030, 16, 1),      # 128-byte ones
    ([2500], 1, 8, 5, 2499, 0, 0),               # rows of one vector, nearly all kept
    ([6000], 3, 8, 16, 1024, 3, 1021),           # three vectors: a slice that ends early
])
def test_moves_in_place_by_slices_of_every_width(pa, lens, KV, D, BLOCK, budget, first, last):
    kc, vc, table, _, ln, w, _ = make(budget, "f16", lens, KV, D, BLOCK)
    want = expect(kc, vc, table, lens, w, budget, first, last, None)
    same(run(pa, kc, vc, table, None, ln, w, budget, first, last), want)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["zeros", "equal", "few", "infs", "nans", "signed", "close"])
@pytest.mark.parametrize("n", [200, 3000, 9000, 40000])
def test_ties_and_odd_weights(pa, n, kind):
    kc, vc, table, dst, ln, w, g = make(n, "f16", [n, n - 1], 1, 64, 16)
    if kind == "zeros":
        w = torch.where(torch.rand(w.shape, generator=g) < 0.7, 0.0, w)
    elif kind == "equal":
        w.fill_(0.25)
    elif kind == "few":
        w = (w * 4).floor()
    elif kind == "infs":
        r = torch.rand(w.shape, generator=g)
        w = torch.where(r < 0.1, torch.inf, torch.where(r > 0.9, -torch.inf, w))
    elif kind == "nans":
        r = torch.rand(w.shape, generator=g)
        w = torch.where(r < 0.6, torch.nan, torch.where(r > 0.9, -torch.inf, w))
    elif kind == "signed":
        w = torch.where(torch.rand(w.shape, generator=g) < 0.5, -w, torch.where(w < 0.1, -0.0, w))
        w[:, ::3] = 0.0
    else:  # all within the last bits of one value
        w = (torch.full_like(w, 1.0).view(torch.int32) + torch.randint(0, 40, w.shape, generator=g, dtype=torch.int32)).view(torch.float32)
    budget = n // 2 + 3
    want = expect(kc, vc, table, [n, n - 1], w, budget, 2, 5, dst)
    same(run(pa, kc, vc, table, dst, ln, w, budget, 2, 5), want)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [16384, 16385, 70000, 131072, 200000])
def test_long_sequences_whose_weights_crowd(pa, n):
    # up to eight CTAs a sequence, and weights read again in every pass past 131072
    kc, vc, table, _, ln, w, g = make(n, "f32", [n, n // 2], 1, 8, 64)
    w = torch.where(torch.rand(w.shape, generator=g) < 0.5, (w * 64).floor() / 64, w)
    budget = n // 3
    want = expect(kc, vc, table, [n, n // 2], w, budget, 3, 100, None)
    same(run(pa, kc, vc, table, None, ln, w, budget, 3, 100), want)


@pytest.mark.gpu
@pytest.mark.parametrize("fresh", [False, True])
def test_pools_past_32_bits_of_offset(pa, fresh):
    # blocks at both ends of pools of 4.8 GB each
    NB, BLOCK, KV, D, n, budget = 150000, 16, 8, 128, 300, 100
    kc = torch.empty(NB, BLOCK, KV, D, dtype=torch.float16, device="cuda")
    vc = torch.empty_like(kc)
    g = torch.Generator().manual_seed(1)
    ids = torch.cat((torch.arange(10), torch.arange(NB - 40, NB)))[torch.randperm(50, generator=g)].to(torch.int32)
    table, dst = ids[:19].view(1, 19).contiguous(), ids[19:26].view(1, 7).contiguous() if fresh else None
    small = torch.randn(2, 50, BLOCK, KV, D, generator=g).half()
    for pool, rows in ((kc, small[0]), (vc, small[1])):
        pool[ids.long().cuda()] = rows.cuda()
    w = torch.rand(1, 19 * BLOCK, generator=g)
    to_small = {int(x): i for i, x in enumerate(ids)}
    local = lambda t: None if t is None else torch.tensor([[to_small[int(x)] for x in t[0]]], dtype=torch.int32)  # noqa: E731
    want = expect(small[0], small[1], local(table), [n], w, budget, 2, 30, local(dst))
    plan = pa.EvictPlan(kc, vc, table.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), w.cuda(), budget=budget,
                        keep_first=2, keep_last=30, dst_table=None if dst is None else dst.cuda())
    new, kept, wout = plan.run()
    torch.cuda.synchronize()
    at = ids.long().cuda()
    same((new.cpu(), kept.cpu(), wout.cpu(), kc[at].cpu(), vc[at].cpu()), want)


@pytest.mark.gpu
def test_bad_lengths_and_blocks_are_reported_and_skipped(pa):
    kc, vc, table, _, ln, w, _ = make(3, "f16", [100, 100, 100], 2, 64, 16)
    cap = table.shape[1] * 16
    ln = torch.tensor([-5, cap + 9, 100], dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = expect(kc, vc, table, [0, cap, 100], w, 60, 1, 1, None)
    same(run(pa, kc, vc, table, None, ln, w, 60, 1, 1, status), want)
    assert int(status) == pa.PA_STATUS_BAD_LENGTH
    # a table entry outside the pool: its rows stay, everything else moves
    lens = [100, 100, 100]
    bad = table.clone()
    bad[1, 2] = kc.shape[0]
    bad[2, 0] = -7
    status.zero_()
    got = run(pa, kc, vc, bad, None, torch.tensor(lens, dtype=torch.int32), w, 60, 1, 1, status)
    assert int(status) == pa.PA_STATUS_BAD_BLOCK
    flat, rows = got[3].view(-1, 2, 64), kc.view(-1, 2, 64).clone()
    for b in range(3):
        ids = kept_of(w[b].numpy(), 100, 60, 1, 1)
        src = kc.view(-1, 2, 64)
        for r, j in enumerate(ids):
            ps, pd = int(bad[b, j // 16]), int(bad[b, r // 16])
            if 0 <= ps < kc.shape[0] and 0 <= pd < kc.shape[0] and r != j:
                rows[pd * 16 + r % 16] = src[ps * 16 + j % 16]
    assert torch.equal(flat, rows)


@pytest.mark.gpu
def test_graph_replay_streams_and_two_plans(pa):
    kc, vc, table, _, ln, w, g = make(9, "bf16", [600, 400, 50], 2, 64, 16)
    d = [x.cuda() for x in (kc, vc, table, ln, w)]
    plan = pa.EvictPlan(*d, budget=100, keep_first=2, keep_last=10)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
    for round_ in range(3):  # other weights, lengths and rows each time
        kc = torch.randn(kc.shape, generator=g).to(kc.dtype)
        w = torch.rand(w.shape, generator=g)
        lens = [600 - 100 * round_, 100 + round_, 90]
        d[0].copy_(kc)
        d[3].copy_(torch.tensor(lens, dtype=torch.int32))
        d[4].copy_(w)
        vc = d[1].cpu()
        graph.replay()
        torch.cuda.synchronize()
        same([x.cpu() for x in (plan.new_lens, plan.kept, plan.weights_out, d[0], d[1])],
             expect(kc, vc, table, lens, w, 100, 2, 10, None))
    # two plans at the same time on two streams, each with its own caches
    other = [x.clone() for x in d]
    other[3].fill_(300)
    want = expect(other[0].cpu(), other[1].cpu(), table, [300] * 3, other[4].cpu(), 77, 0, 0, None)
    want1 = expect(d[0].cpu(), d[1].cpu(), table, d[3].tolist(), d[4].cpu(), 100, 2, 10, None)
    plan2 = pa.EvictPlan(*other, budget=77)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    plan.run(s1)
    plan2.run(s2)
    torch.cuda.synchronize()
    same([x.cpu() for x in (plan2.new_lens, plan2.kept, plan2.weights_out, other[0], other[1])], want)
    same([x.cpu() for x in (plan.new_lens, plan.kept, plan.weights_out, d[0], d[1])], want1)


@pytest.mark.gpu
def test_refused_arguments(pa):
    kc, vc, table, _, ln, w, _ = make(9, "bf16", [60], 2, 64, 16)
    d = [x.cuda() for x in (kc, vc, table, ln, w)]
    with pytest.raises(ValueError):
        pa.EvictPlan(*d, budget=0)
    with pytest.raises(ValueError):
        pa.EvictPlan(*d[:4], d[4][:, :-1], budget=10)
    with pytest.raises(ValueError):
        pa.EvictPlan(*d[:4], d[4].double(), budget=10)
    with pytest.raises(TypeError):
        pa.EvictPlan(*d[:2], d[2].long(), *d[3:], budget=10)
    with pytest.raises(pa.PagedAttentionError):
        pa.EvictPlan(*d, budget=10, keep_first=6, keep_last=5).run()
    with pytest.raises(pa.PagedAttentionError):
        pa.EvictPlan(*d, budget=10, weights_out=d[4]).run()
