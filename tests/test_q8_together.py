"""The operators of the cache in 8 bits as they are used together: a serving
loop (blocks planned, positions turned, rows stored, blocks selected, attended
to, sequences ended and replaced), against plain arithmetic on the host; the
same captured in a graph and replayed; two loops on streams of their own; calls
on a stream that is not torch's current one; the sizes at the limits."""
import math

import numpy as np
import pytest
import torch

from test_one_call_streams import while_the_current_stream_is_busy
from test_q8 import DT, Cache, as64, ints, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_182_gb300 import binding

    return binding


class Loop:
    """Device state of a serving loop and the calls of one step; every sequence gets up to N rows a step."""

    def __init__(self, pa, B=5, H=8, KV=2, D=64, BLOCK=8, maxb=24, pool=90, N=20, budget=6, fmt="f16", seed=0):
        self.pa, self.B, self.N, self.BLOCK, self.fmt, self.pool = pa, B, N, BLOCK, fmt, pool
        g = torch.Generator().manual_seed(seed)
        self.c = c = Cache(seed, [1] * B, KV, D, BLOCK, width=maxb, spare=pool - B * maxb if pool > B * maxb else 0)
        c.lens = np.zeros(B, np.int32)
        c.table = np.full((B, maxb), -1, np.int32)
        c.kc, c.vc = (np.zeros((pool, BLOCK, KV, D), np.int8) for _ in range(2))
        c.ks, c.vs = (np.zeros((pool, KV), np.float32) for _ in range(2))
        c.bounds = np.zeros((pool, KV, 2, D), np.int8)
        self.dev = c.cuda()
        self.kc, self.vc, self.ks, self.vs, self.table = self.dev
        self.bounds = torch.from_numpy(c.bounds.copy()).cuda()
        self.lens, self.add, self.keep = (ints([0] * B) for _ in range(3))
        self.free, self.count, self.status = torch.randperm(pool, generator=g).to(torch.int32).cuda(), ints([pool]), ints([0])
        dt = DT[fmt]
        self.q = torch.zeros(B, H, N, D, dtype=dt, device="cuda")
        self.k, self.v = (torch.zeros(B, KV, N, D, dtype=dt, device="cuda") for _ in range(2))
        self.scale = float(np.float32(D ** -0.5))
        self.plan = pa.BlockPlan(self.table, self.lens, self.free, self.count, BLOCK=BLOCK, width=N, add=self.add, keep=self.keep,
                                 status=self.status)
        self.rot = pa.rotary_table(D)
        self.turn = pa.RotaryPlan(self.q, self.k, self.plan.positions, self.rot)
        self.store = pa.Q8AppendPlan(self.turn.k_out, self.v, *self.dev[:4], self.table, self.keep, counts=self.add, bounds=self.bounds,
                                     status=self.status)
        # (the last row's attention: of up to 16 rows a call, the step looks at one)
        self.last = torch.zeros(B, H, 1, D, dtype=dt, device="cuda")
        self.pick = pa.Q8SelectPlan(self.last, self.bounds, self.ks, self.table, self.plan.new_lens, BLOCK=BLOCK, budget=budget,
                                    keep_first=1, keep_last=2, status=self.status)
        self.sparse = pa.Q8Plan(self.last, *self.dev, self.plan.new_lens, scale=self.scale, causal=True, selected=self.pick.selected,
                                counts=self.pick.counts, status=self.status)
        self.full = pa.Q8Plan(self.last, *self.dev, self.plan.new_lens, scale=self.scale, causal=True, status=self.status)

    def step(self):
        """One step of every sequence; every call is asynchronous on the current stream."""
        self.plan.run()
        self.turn.run()
        self.store.run()
        at = (self.add.long() - 1).clamp(min=0).view(-1, 1, 1, 1).expand(-1, self.q.shape[1], 1, self.q.shape[3])
        self.last.copy_(self.turn.q_out.gather(2, at))
        self.pick.run()
        out = self.sparse.run(), self.full.run()
        self.lens.copy_(self.plan.new_lens)
        self.count.copy_(self.plan.new_free_count)
        return out


def inputs(loop, rng, n):
    """Rows of a step, and which sequences end, go on, or begin."""
    lens = loop.lens.cpu().numpy()
    done = (rng.random(loop.B) < 0.12) | (lens > 140)
    keep = np.where(done, 0, lens)
    add = np.where(keep == 0, rng.integers(0, loop.N + 1, loop.B), rng.integers(0, 4, loop.B))
    rows = [torch.from_numpy(rng.normal(0, s, t.shape).astype(np.float32)).to(t.dtype) for t, s in ((loop.q, 2), (loop.k, 1), (loop.v, 1))]
    return keep, add, rows


def feed(loop, keep, add, rows):
    loop.keep.copy_(ints(keep)), loop.add.copy_(ints(add))
    for t, r in zip((loop.q, loop.k, loop.v), rows):
        t.copy_(r)


@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
def test_serving_loop(pa, fmt):
    loop, rng = Loop(pa, fmt=fmt, seed=3), np.random.default_rng(5)
    c = loop.c
    for n in range(45):
        keep, add, rows = inputs(loop, rng, n)
        feed(loop, keep, add, rows)
        sparse, full = loop.step()
        torch.cuda.synchronize()
        assert int(loop.status) == 0
        new = loop.lens.cpu().numpy()
        np.testing.assert_array_equal(new, keep + add)
        # every block belongs to one sequence or is free
        c.table = loop.table.cpu().numpy()
        used = np.concatenate([c.table[b, : -(-int(new[b]) // loop.BLOCK)] for b in range(loop.B)] + [loop.free[: int(loop.count)].cpu().numpy()])
        assert sorted(used) == list(range(loop.pool))
        # the store, from what the rotation gave
        c.lens = keep.astype(np.int32)
        c.append(loop.turn.k_out.float().cpu().numpy(), rows[1 + 1].float().numpy(), add, True)
        for name, g, w in (("kc", loop.kc, c.kc), ("vc", loop.vc, c.vc), ("ks", loop.ks, c.ks), ("vs", loop.vs, c.vs)):
            for b in range(loop.B):
                held = c.table[b, : -(-int(new[b]) // loop.BLOCK)]
                np.testing.assert_array_equal(g[held.tolist()].cpu().numpy(), w[held], err_msg=name)
        c.lens = new.astype(np.int32)
        want = c.select(loop.last.float().cpu().numpy(), 6, 1, 2)
        np.testing.assert_array_equal(loop.pick.selected.cpu().numpy(), want[0])
        np.testing.assert_array_equal(loop.pick.counts.cpu().numpy(), want[1])
        for got, sel in ((full, (None, None)), (sparse, want)):
            y, tol = c.attend(as64(loop.last), loop.scale, True, fmt, *sel)
            assert np.all(np.abs(as64(got) - y) <= tol), n


def test_the_step_in_a_graph(pa):
    a, b, rng = Loop(pa, seed=4), Loop(pa, seed=4), np.random.default_rng(6)
    steps = []
    for n in range(12):
        steps.append(inputs(a, rng, n))
        feed(a, *steps[-1])
        steps[-1] += (tuple(t.clone() for t in a.step()), a.lens.clone(), a.kc.clone(), a.bounds.clone(), a.table.clone())
        torch.cuda.synchronize()
    feed(b, np.zeros(b.B), np.zeros(b.B), steps[0][2])
    b.step()  # (workspaces, modules: before the capture)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.step()
    for keep, add, rows, want, lens, kc, bounds, table in steps:
        feed(b, keep, add, rows)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((*want, lens, kc, bounds, table), (*out, b.lens, b.kc, b.bounds, b.table)):
            assert torch.equal(x, y)


def test_two_loops_on_streams_of_their_own(pa):
    kinds = (dict(seed=7, fmt="bf16"), dict(seed=8, B=9, D=128, KV=4, BLOCK=16, maxb=12, pool=110, budget=4))
    loops = [Loop(pa, **k) for k in kinds]
    rngs = [np.random.default_rng(9 + i) for i in range(2)]
    steps, want = [[], []], [[], []]
    for n in range(15):
        for i, loop in enumerate(loops):
            steps[i].append(inputs(loop, rngs[i], n))
            feed(loop, *steps[i][-1])
            want[i].append([t.clone() for t in loop.step()])
            torch.cuda.synchronize()
    end = [(x.lens.clone(), x.kc.clone(), x.vs.clone(), x.free[: int(x.count)].clone()) for x in loops]
    loops = [Loop(pa, **k) for k in kinds]
    ready = [[[ints(s[0]), ints(s[1]), [r.cuda() for r in s[2]]] for s in steps[i]] for i in range(2)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for n in range(15):
        for i, loop in enumerate(loops):
            with torch.cuda.stream(streams[i]):
                keep, add, rows = ready[i][n]
                loop.keep.copy_(keep), loop.add.copy_(add)
                for t, r in zip((loop.q, loop.k, loop.v), rows):
                    t.copy_(r)
                got[i].append([t.clone() for t in loop.step()])
    torch.cuda.synchronize()
    for i, loop in enumerate(loops):
        for x, y in zip(want[i], got[i]):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
        for x, y in zip(end[i], (loop.lens, loop.kc, loop.vs, loop.free[: int(loop.count)])):
            assert torch.equal(x, y)


def test_calls_on_another_stream(pa):
    c = Cache(22, [3000, 40, 700], 2, 128, 16, more=20)
    q, kn = rows_of(c.rng, "f16", 3, 8, 1, 128).cuda(), rows_of(c.rng, "f16", 3, 2, 5, 128).cuda()
    kc, vc, ks, vs, table = c.cuda()
    lens, bounds = ints(c.lens), torch.from_numpy(c.bounds).cuda()
    free, count = ints(np.arange(500) + 10), ints([400])
    calls = [
        lambda s: pa.decode_q8(q, kc, vc, ks, vs, table, lens, scale=0.09, stream=s),
        lambda s: pa.select_blocks_q8(q, bounds, ks, table, lens, BLOCK=16, budget=20, stream=s),
        lambda s: pa.cache_read_q8(kc, vc, ks, vs, table, ints([0, 3, 100]), width=40, counts=ints([40, 30, 40]), stream=s),
        lambda s: pa.cache_append_q8(kn, kn, kc, vc, ks, vs, table, lens, stream=s),
        lambda s: pa.plan_blocks(table.clone(), lens, free, count, BLOCK=16, width=1, stream=s),
    ]
    need = pa.q8_workspace_bytes(3, 8, 2, 128, 1)
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        want = [t.clone() for t in (want if isinstance(want, tuple) else (want,))]
        for _ in range(2):
            for a, b in zip(want, while_the_current_stream_is_busy(call, need, q.numel() * 2, 2 * 3 * 2 * 40 * 128, 240, 12, 4)):
                assert torch.equal(a, b)


def test_a_workspace_of_ones_own_serves_calls_in_turn(pa):
    """Shapes with other passes and splits share one; each leaves it as the next needs it."""
    need = max(pa.q8_workspace_bytes(*s) for s in ((3, 8, 2, 128, 1), (3, 16, 2, 64, 4), (40, 8, 2, 128, 1)))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    cases = []
    for lens, H, D, NQ, fmt in (([9000, 40, 700], 8, 128, 1, "f16"), ([9000, 40, 700], 16, 64, 4, "f32"), ([500] * 40, 8, 128, 1, "bf16")):
        c = Cache(23, lens, 2, D, 16)
        q = rows_of(c.rng, fmt, len(lens), H, NQ, D).cuda()
        dev = c.cuda()
        own = pa.decode_q8(q, *dev, ints(lens), scale=0.1, causal=True)
        cases.append((pa.Q8Plan(q, *dev, ints(lens), scale=0.1, causal=True, workspace=ws), own))
    for _ in range(3):
        for plan, own in cases:
            got = plan.run().clone()
            assert torch.equal(got, own)


# ------------------------------------------------------------------ sizes at the limits
def test_many_short_sequences(pa):
    """4096 sequences: the schedule's limit, a few tokens each."""
    B, KV, D, BLOCK = 4096, 1, 64, 8
    c = Cache(24, [1] * B, KV, D, BLOCK, width=3)
    c.lens = c.rng.integers(0, 25, B).astype(np.int32)
    q = rows_of(c.rng, "f16", B, 2, 1, D)
    dev = c.cuda()
    out = pa.decode_q8(q.cuda(), *dev, ints(c.lens), scale=0.125)
    sel, cnt = pa.select_blocks_q8(q.cuda(), torch.from_numpy(c.bounds).cuda(), dev[2], dev[4], ints(c.lens), BLOCK=BLOCK, budget=2, keep_last=1)
    few = pa.decode_q8(q.cuda(), *dev, ints(c.lens), scale=0.125, selected=sel, counts=cnt)
    torch.cuda.synchronize()
    want, tol = c.attend(as64(q), 0.125, False, "f16")
    assert np.all(np.abs(as64(out) - want) <= tol)
    ws, wc = c.select(q.float().numpy(), 2, 0, 1)
    np.testing.assert_array_equal(sel.cpu().numpy(), ws)
    want, tol = c.attend(as64(q), 0.125, False, "f16", ws, wc)
    assert np.all(np.abs(as64(few) - want) <= tol)


@pytest.mark.parametrize("fmt", ["f32", "f16"])
def test_one_warp_over_many_tokens(pa, fmt):
    """As many segments as CTAs several times over: each warp adds up thousands of tokens."""
    B, D, BLOCK, n = 320, 64, 16, 6000
    per = -(-n // BLOCK)
    g = torch.Generator().manual_seed(1)
    kc, vc = (torch.randint(-127, 128, (per * 4, BLOCK, 1, D), generator=g, dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.rand(per * 4, 1, generator=g) * 0.01 + 0.001 for _ in range(2))
    table = torch.stack([torch.randperm(per * 4, generator=g)[:per] for _ in range(B)]).to(torch.int32)
    q = torch.randn(B, 4, 1, D, generator=g).to(DT[fmt])
    out = pa.decode_q8(q.cuda(), kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda(), table.cuda(), ints([n] * B), scale=0.125)
    torch.cuda.synchronize()
    c = Cache(0, [n] * B, 1, D, BLOCK)
    c.kc, c.vc, c.ks, c.vs, c.table = (t.numpy() for t in (kc, vc, ks, vs, table))
    for b in (0, 1, 100, 151, 152, 319):
        c.lens, c.table = np.array([n], np.int32), table[b: b + 1].numpy()
        want, tol = c.attend(as64(q[b: b + 1]), 0.125, False, fmt)
        assert np.all(np.abs(as64(out[b: b + 1]) - want) <= tol), b


def test_the_most_query_rows(pa):
    """64 heads of 16 rows on one KV head: 1024 rows a head, in passes."""
    for fmt in ("f16", "f32"):
        c = Cache(25, [200, 20, 7], 1, 64, 16)
        q = rows_of(c.rng, fmt, 3, 64, 16, 64)
        dev = c.cuda()
        out = pa.decode_q8(q.cuda(), *dev, ints(c.lens), scale=0.125, causal=True)
        sel, cnt = pa.select_blocks_q8(q.cuda(), torch.from_numpy(c.bounds).cuda(), dev[2], dev[4], ints(c.lens), BLOCK=16, budget=5, keep_last=2)
        torch.cuda.synchronize()
        want, tol = c.attend(as64(q), 0.125, True, fmt)
        assert np.all(np.abs(as64(out) - want) <= tol)
        ws, wc = c.select(q.float().numpy(), 5, 0, 2)
        np.testing.assert_array_equal(sel.cpu().numpy(), ws)
        np.testing.assert_array_equal(cnt.cpu().numpy(), wc)


@pytest.mark.parametrize("B,KV,D,R", [(1, 1, 128, 5), (40, 8, 128, 4), (2, 2, 64, 200), (40, 8, 64, 40)])
def test_selection_over_the_longest_table(pa, B, KV, D, R):
    """32768 blocks a row (most of them shared here), clusters or one CTA a head, rows in parts."""
    maxb, pool = 32768, 300
    g = torch.Generator().manual_seed(2)
    bounds = torch.randint(-127, 128, (pool, KV, 2, D), generator=g, dtype=torch.int8).sort(2).values
    ks = torch.rand(pool, KV, generator=g)
    table = torch.randint(0, pool, (B, maxb), generator=g).to(torch.int32)
    lens = torch.full((B,), 100, dtype=torch.int32)
    lens[0], lens[-1] = maxb * 8, maxb * 8 - 1003
    q = torch.randn(B, KV * R if R <= 40 else KV * (R // 10), 1 if R <= 40 else 10, D, generator=g)
    sel, cnt = pa.select_blocks_q8(q.cuda(), bounds.cuda(), ks.cuda(), table.cuda(), lens.cuda(), BLOCK=8, budget=700, keep_first=3, keep_last=5)
    torch.cuda.synchronize()
    c = Cache(0, [8] * B, KV, D, 8)
    c.bounds, c.ks = bounds.numpy(), ks.numpy()
    for b in {0, B - 1}:
        c.lens, c.table = lens[b: b + 1].numpy(), table[b: b + 1].numpy()
        ws, wc = c.select(q[b: b + 1].numpy(), 700, 3, 5)
        np.testing.assert_array_equal(sel[b].cpu().numpy(), ws[0])
        np.testing.assert_array_equal(cnt[b].cpu().numpy(), wc[0])


@pytest.mark.parametrize("maxb,D,R,KV", [(32512, 128, 64, 1), (32480, 128, 300, 1), (30000, 64, 128, 30)])
def test_selection_where_shared_memory_is_full(pa, maxb, D, R, KV):
    """Tables whose scores leave room for some of the rows at a time, to the last bytes."""
    g = torch.Generator().manual_seed(3)
    pool, c = 200, Cache(0, [8], KV, D, 8)
    c.bounds = torch.randint(-127, 128, (pool, KV, 2, D), generator=g, dtype=torch.int8).sort(2).values.numpy()
    c.ks = torch.rand(pool, KV, generator=g).numpy()
    c.table = torch.randint(0, pool, (1, maxb), generator=g).to(torch.int32).numpy()
    c.lens = np.array([1500], np.int32)
    q = torch.randn(1, KV * (R if R <= 128 else R // 10), 1 if R <= 128 else 10, D, generator=g)
    sel, cnt = pa.select_blocks_q8(q.cuda(), torch.from_numpy(c.bounds).cuda(), torch.from_numpy(c.ks).cuda(),
                                   torch.from_numpy(c.table).cuda(), ints(c.lens), BLOCK=8, budget=60)
    torch.cuda.synchronize()
    ws, wc = c.select(q.numpy(), 60, 0, 1)
    np.testing.assert_array_equal(sel.cpu().numpy(), ws)
    np.testing.assert_array_equal(cnt.cpu().numpy(), wc)


@pytest.mark.parametrize("op", ["blocks", "append", "read", "select", "decode"])
def test_a_decode_that_reads_its_inputs_early_behind_them(pa, op):
    """A decode with inputs_unchanged: the kernel ahead of it writes none of its inputs, the one before that its q."""
    from test_scored import make

    x, _ = make(41, "f16", [6000, 5000, 300], 16, 2, 128, 16, 1)
    first = pa.Plan(*x, scale=0.09, causal=True)
    second = pa.Plan(first.out, *x[1:], scale=1.0, causal=True, inputs_unchanged=True)
    c = Cache(29, [40, 3], 2, 64, 16, more=8)
    dev, lens = c.cuda(), ints(c.lens)
    rows, q = rows_of(c.rng, "f16", 2, 2, 2, 64).cuda(), rows_of(c.rng, "f16", 2, 4, 1, 64).cuda()
    between = {"blocks": lambda: pa.BlockPlan(dev[4], lens, ints(range(8)), ints([8]), BLOCK=16, width=1),
               "append": lambda: pa.Q8AppendPlan(rows, rows, *dev, lens),
               "read": lambda: pa.Q8ReadPlan(*dev, ints([0, 0]), width=4),
               "select": lambda: pa.Q8SelectPlan(q, torch.from_numpy(c.bounds).cuda(), dev[2], dev[4], lens, BLOCK=16, budget=2),
               "decode": lambda: pa.Q8Plan(q, *dev, lens, scale=0.125)}[op]()
    sets = [torch.randn_like(x[0]) for _ in range(2)]
    want = []
    for s in sets:
        x[0].copy_(s)
        first.run()
        torch.cuda.synchronize()
        want.append(second.run().clone())
        torch.cuda.synchronize()
    assert not torch.equal(*want)
    got = []
    for n in range(40):
        x[0].copy_(sets[n % 2])
        first.run()
        between.run()
        got.append(second.run().clone())
    torch.cuda.synchronize()
    for n, t in enumerate(got):
        assert torch.equal(t, want[n % 2]), n


def test_rows_that_are_one_row(pa):
    """New rows broadcast over sequences and tokens (strides of zero), and many heads."""
    c = Cache(26, [0, 13], 3, 64, 16, more=20)
    kn = rows_of(c.rng, "bf16", 1, 3, 1, 64).cuda().expand(2, 3, 20, 64)
    dev = c.cuda()
    pa.cache_append_q8(kn, kn, *dev, ints(c.lens))
    torch.cuda.synchronize()
    x = kn.float().cpu().numpy()
    c.append(x, x, [20, 20], False)
    for g, w in zip(dev, (c.kc, c.vc, c.ks, c.vs)):
        np.testing.assert_array_equal(g.cpu().numpy(), w)


def test_no_sequence_and_no_row(pa):
    c = Cache(27, [5], 2, 64, 16)
    kc, vc, ks, vs, _ = c.cuda()
    none = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    lens = torch.zeros(0, dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 4, 1, 64, device="cuda").half()
    k = torch.zeros(0, 2, 3, 64, device="cuda").half()
    assert pa.decode_q8(q, kc, vc, ks, vs, none, lens, scale=0.1).shape == q.shape
    assert pa.select_blocks_q8(q, torch.from_numpy(c.bounds).cuda(), ks, none, lens, BLOCK=16, budget=3)[0].shape == (0, 2, 3)
    assert pa.cache_read_q8(kc, vc, ks, vs, none, lens, width=3)[0].shape == (0, 2, 3, 64)
    pa.cache_append_q8(k, k, kc, vc, ks, vs, none, lens)
    one = torch.zeros(1, 2, 0, 64, device="cuda").half()
    pa.cache_append_q8(one, one, kc, vc, ks, vs, ints([[0]]), ints([5]))
    assert pa.cache_read_q8(kc, vc, ks, vs, ints([[0]]), ints([5]), width=0)[0].shape == (1, 2, 0, 64)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(kc.cpu().numpy(), c.kc)


def test_a_long_prompt(pa):
    """65536 rows in one call, as many as a prompt may have."""
    KV, D, BLOCK, N = 1, 64, 64, 65536
    nb = N // BLOCK + 1
    g = torch.Generator().manual_seed(4)
    kn, vn = (torch.randn(1, KV, N, D, generator=g).half().cuda() for _ in range(2))
    kc, vc = (torch.zeros(nb, BLOCK, KV, D, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(nb, KV, device="cuda") for _ in range(2))
    table = torch.randperm(nb, generator=g).to(torch.int32).view(1, nb).cuda()
    pa.cache_append_q8(kn, vn, kc, vc, ks, vs, table, ints([0]))
    ko, vo = pa.cache_read_q8(kc, vc, ks, vs, table, ints([0]), width=N, dtype=torch.float32)
    torch.cuda.synchronize()
    for x, y in ((kn, ko), (vn, vo)):
        rows = x.float().view(N // BLOCK, BLOCK * D)
        scale = (rows.abs().amax(1, keepdim=True).double() / 127).float()
        want = (rows.double() / scale.double()).round().clamp(-127, 127).float() * scale
        assert torch.equal(y.view(N // BLOCK, BLOCK * D), want)
    q = torch.randn(1, 4, 1, D, generator=g).half().cuda()
    out = pa.decode_q8(q, kc, vc, ks, vs, table, ints([N]), scale=0.125)
    s = torch.softmax(q.double().view(4, D) @ ko.double().view(N, D).T * 0.125, -1)
    want = (s @ vo.double().view(N, D)).view(out.shape)
    # (scores off by 2^-16 of their parts, weights by 2^-11, sums and the result by as much again)
    bound = (math.log(2) * 2 * (0.125 * 1.4427 * float((q.double().view(4, D).abs() @ ko.double().view(N, D).abs().T).max()) * D * 2.0 ** -23
                                + 2.0 ** -20 * 60) + 2.0 ** -11 + 2.0 ** -13) * (s @ vo.double().view(N, D).abs()).view(out.shape)
    assert bool(((out.double() - want).abs() <= bound + 2.0 ** -11 * want.abs() + 2.0 ** -25).all())
