"""Sequences that the block plan refuses, and the store behind it: `kept` and
`granted` are what the store may be given, and no block of another sequence
changes by a byte."""
import numpy as np
import pytest
import torch

from test_blocks import A, ALIGN, DIMS, call, check, expect, state
from test_q8 import Cache, as64, ints, rows_of
from test_q8_together import Loop, feed


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_182_gb300 import _build

    _build.build()
    from paged_kv_cache_182_gb300 import binding

    return binding


@pytest.mark.parametrize("kw,code", [
    (dict(kept=9 * A + 2), ALIGN), (dict(granted=9 * A + 1), ALIGN), (dict(kept=9 * A, granted=9 * A + 4), DIMS),
    (dict(kept=5 * A), DIMS), (dict(granted=2 * A), DIMS), (dict(add=9 * A, granted=9 * A), DIMS), (dict(keep=9 * A, kept=9 * A), DIMS),
])
def test_refusals(pa, kw, code):
    assert call(pa, **kw) == code


def split(table, lens, stack, count, BLOCK, N, **kw):
    """(kept, granted) by the plain plan: a sequence that was refused has its length and no slot."""
    new, slots, pos = expect(table, lens, stack, count, BLOCK, N, **kw)[2], *expect(table, lens, stack, count, BLOCK, N, **kw)[4:6]
    granted = (pos >= 0).sum(1) if "starts" not in kw else (slots >= 0).sum(1)
    return new - granted, granted


def plan_of(pa, table, lens, stack, count, BLOCK, N, **kw):
    plan = pa.BlockPlan(ints(table), ints(lens), ints(stack), ints([count]), BLOCK=BLOCK, width=N, **{k: ints(v) for k, v in kw.items()})
    plan.kept.fill_(-99), plan.granted.fill_(-99)
    return plan


@pytest.mark.gpu
@pytest.mark.parametrize("spare", [0, 1, 2, 3, 5, 9])
def test_kept_and_granted(pa, spare):
    """Refused for want of blocks, for the table's width, shortened, done, and with values out of range."""
    lens, add, keep = [16, 16, 10, 64, 16, 40, 127, 33, 0], [1, 20, 2, 70, 33, 0, 5, 99, -3], [16, 3, 10, 64, 0, 12, 127, 50, -1]
    x = state(3, lens, 16, 8, spare)
    want = split(*x, 16, 70, add=add, keep=keep)
    for _ in range(2):
        plan = plan_of(pa, *x, 16, 70, add=add, keep=keep)
        new = plan.run()[0]
        kept, granted = torch.empty_like(new), torch.empty_like(new)
        pa.plan_blocks(*(ints(t) for t in x[:3]), ints([x[3]]), BLOCK=16, width=70, add=ints(add), keep=ints(keep), kept=kept, granted=granted)
        torch.cuda.synchronize()
        for k, g in ((plan.kept, plan.granted), (kept, granted)):
            np.testing.assert_array_equal(k.cpu().numpy(), want[0])
            np.testing.assert_array_equal(g.cpu().numpy(), want[1])
            assert torch.equal(k + g, new)


@pytest.mark.gpu
@pytest.mark.parametrize("BLOCK", [2 ** 30 - 1, 2 ** 29, 2 ** 29 - 3])
def test_the_largest_blocks(pa, BLOCK):
    """Lengths whose sum with a block passes 2^31."""
    maxb = (2 ** 30 - 1) // BLOCK
    pool = (2 ** 31 - 1) // BLOCK
    lens = np.array([maxb * BLOCK, maxb * BLOCK, 0][: pool + 1])
    table = np.arange(len(lens) * maxb).reshape(len(lens), maxb) % pool
    for N, keep in ((1, [0, 1, 0]), (70, [maxb * BLOCK, maxb * BLOCK - 70, 0]), (65536, [maxb * BLOCK - 65535, 5, 0])):
        check(pa, table, lens, np.full(pool, -1), 0, BLOCK, N, add=[N] * len(lens), keep=keep[: len(lens)], again=False)


@pytest.mark.gpu
def test_refused_tensors(pa):
    x = state(3, [16, 5], 16, 8, 4)
    good = dict(block_table=ints(x[0]), seq_lens=ints(x[1]), free_blocks=ints(x[2]), free_count=ints([x[3]]), BLOCK=16, width=2)
    for name in ("kept", "granted"):
        for bad in (ints([0]), ints([0, 0]).long(), ints([0, 0]).cpu(), ints([0, 0, 0, 0])[::2]):
            with pytest.raises(ValueError):
                pa.plan_blocks(**good, **{name: bad})
        with pytest.raises(pa.PagedAttentionError):
            pa.plan_blocks(**good, **{name: good["seq_lens"]})


@pytest.mark.gpu
def test_a_refused_sequence_stores_nothing(pa):
    """A gives two of its blocks back, B takes them, then A asks for more than there is: A's table still names B's blocks."""
    c = Cache(40, [40, 0], 2, 64, 16, width=3)
    c.table = np.array([[0, 1, 2], [-1, -1, -1]], np.int32)
    dev, bounds, status = c.cuda(), torch.from_numpy(c.bounds.copy()).cuda(), ints([0])
    free, count, lens = ints([-1] * 3), ints([0]), ints(c.lens)
    kn, vn = (rows_of(c.rng, "f16", 2, 2, 40, 64) for _ in range(2))
    for keep, add, says in (([10, 0], [0, 32], 0), ([10, 32], [10, 0], 16), ([4, 32], [20, 0], 16)):
        plan = pa.BlockPlan(dev[4], lens, free, count, BLOCK=16, width=40, add=ints(add), keep=ints(keep), status=status)
        plan.run()
        pa.cache_append_q8(kn.cuda(), vn.cuda(), *dev, plan.kept, counts=plan.granted, bounds=bounds, status=status)
        torch.cuda.synchronize()
        assert int(status) == says
        if not says:
            c.table, c.lens = dev[4].cpu().numpy(), np.array(keep, np.int32)
            c.append(kn.float().numpy(), vn.float().numpy(), add, True)
        for g, w in zip((*dev[:4], bounds), (c.kc, c.vc, c.ks, c.vs, c.bounds)):
            np.testing.assert_array_equal(g.cpu().numpy(), w)
        lens, count = plan.new_lens.clone(), plan.new_free_count.clone()
        assert lens.tolist() == [10, 32]
        status.zero_()


class Tight(Loop):
    """The serving loop with the store behind the plan's own counts, and a pool that is too small."""

    def __init__(self, pa, **kw):
        super().__init__(pa, pool=11, **kw)
        self.store = pa.Q8AppendPlan(self.turn.k_out, self.v, *self.dev[:4], self.table, self.plan.kept, counts=self.plan.granted,
                                     bounds=self.bounds, status=self.status)

    def step(self):
        """As Loop.step, for counts outside [0, N] too: the row looked at is one that is there."""
        self.plan.run()
        self.turn.run()
        self.store.run()
        at = (self.add.long() - 1).clamp(0, self.N - 1).view(-1, 1, 1, 1).expand(-1, self.q.shape[1], 1, self.q.shape[3])
        self.last.copy_(self.turn.q_out.gather(2, at))
        self.pick.run()
        out = self.sparse.run(), self.full.run()
        self.lens.copy_(self.plan.new_lens)
        self.count.copy_(self.plan.new_free_count)
        return out


def asked(loop, rng):
    """What the sequences ask for: more rows, fewer tokens, both; now and then what the plan has to clamp."""
    n = loop.lens.cpu().numpy()
    u = rng.random((2, loop.B))
    keep = np.where((u[0] < 0.15) | (n > 120), 0, np.where(u[0] < 0.35, n // 2, np.where(u[0] < 0.4, n + 5, n)))
    add = np.where(u[1] < 0.7, rng.integers(0, 4, loop.B), rng.integers(0, loop.N + 4, loop.B))
    rows = [torch.from_numpy(rng.normal(0, s, t.shape).astype(np.float32)).to(t.dtype) for t, s in ((loop.q, 2), (loop.k, 1), (loop.v, 1))]
    return keep, add, rows


@pytest.mark.gpu
def test_a_loop_with_too_few_blocks(pa):
    loop, rng, refused = Tight(pa, seed=12), np.random.default_rng(13), 0
    c = loop.c
    for n in range(60):
        keep, add, rows = asked(loop, rng)
        feed(loop, keep, add, rows)
        before = [t.cpu().numpy().astype(np.int64) for t in (loop.table, loop.lens, loop.free)]
        loop.status.zero_()
        want = expect(*before, int(loop.count), loop.BLOCK, loop.N, add=add, keep=keep)
        kept, granted = split(*before, int(loop.count), loop.BLOCK, loop.N, add=add, keep=keep)
        sparse, full = loop.step()
        torch.cuda.synchronize()
        refused += want[6] >> 4 & 1
        assert int(loop.status) == want[6]
        for g, w in zip((loop.table, loop.free, loop.lens, loop.count, loop.plan.kept, loop.plan.granted), (*want[:4], kept, granted)):
            np.testing.assert_array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
        new = loop.lens.cpu().numpy()
        c.table = loop.table.cpu().numpy()
        used = np.concatenate([c.table[b, : -(-int(new[b]) // loop.BLOCK)] for b in range(loop.B)] + [loop.free[: int(loop.count)].cpu().numpy()])
        assert sorted(used) == list(range(loop.pool))
        # the whole pool, byte for byte
        c.lens = kept.astype(np.int32)
        c.append(loop.turn.k_out.float().cpu().numpy(), rows[2].float().numpy(), granted, True)
        for g, w in zip((loop.kc, loop.vc, loop.ks, loop.vs, loop.bounds), (c.kc, c.vc, c.ks, c.vs, c.bounds)):
            np.testing.assert_array_equal(g.cpu().numpy(), w)
        c.lens = new.astype(np.int32)
        y, tol = c.attend(as64(loop.last), loop.scale, True, "f16")
        assert np.all(np.abs(as64(full) - y) <= tol), n
    assert refused > 10


@pytest.mark.gpu
def test_two_plans_in_turn(pa):
    """A loop without copies: each plan's lengths and count are what the other one left."""
    rng = np.random.default_rng(16)
    table, lens, stack, count = state(17, [40, 3, 0, 17], 8, 12, 9)
    t, s, n, c, add, keep = ints(table), ints(stack), ints(lens), ints([count]), ints([0] * 4), ints([0] * 4)
    one = pa.BlockPlan(t, n, s, c, BLOCK=8, width=20, add=add, keep=keep)
    two = pa.BlockPlan(t, one.new_lens, s, one.new_free_count, BLOCK=8, width=20, add=add, keep=keep, new_lens=n, new_free_count=c)
    for step in range(30):
        k = np.where(rng.random(4) < 0.2, lens // 3, lens)
        a = rng.integers(0, 21, 4) * (rng.random(4) < 0.5)
        add.copy_(ints(a)), keep.copy_(ints(k))
        new, left, slots, pos = (one, two)[step % 2].run()
        torch.cuda.synchronize()
        want = expect(table, lens, stack, count, 8, 20, add=a, keep=k)
        table, stack, lens, count = want[:4]
        for g, w in zip((t, s, new, left, slots, pos), want):
            np.testing.assert_array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))


@pytest.mark.gpu
def test_a_refusal_in_a_graph(pa):
    a, b, rng = Tight(pa, seed=14), Tight(pa, seed=14), np.random.default_rng(15)
    steps, refused = [], 0
    for n in range(25):
        steps.append(asked(a, rng))
        feed(a, *steps[-1])
        a.status.zero_()
        steps[-1] += ([t.clone() for t in (*a.step(), a.lens, a.plan.kept, a.plan.granted, a.kc, a.vc, a.ks, a.vs, a.bounds, a.table, a.status)],)
        torch.cuda.synchronize()
        refused += int(a.status) >> 4 & 1
    assert refused > 3
    feed(b, np.zeros(b.B), np.zeros(b.B), steps[0][2])
    b.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.step()
    for keep, add, rows, want in steps:
        feed(b, keep, add, rows)
        b.status.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, (*out, b.lens, b.plan.kept, b.plan.granted, b.kc, b.vc, b.ks, b.vs, b.bounds, b.table, b.status)):
            assert torch.equal(x, y)
