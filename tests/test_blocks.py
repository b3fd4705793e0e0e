"""Block tables and slots of a step (include/pa_blocks.h): refusals on the CPU,
plans on the GPU against a plain list of blocks.  Whole numbers throughout:
every comparison is exact."""
import ctypes

import numpy as np
import pytest
import torch

A = 1 << 24
NULL, DIMS, UNSUP, ALIGN = -1, -2, -3, -4


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_182_gb300 import _build

    _build.build()
    from paged_kv_cache_182_gb300 import binding

    return binding


# ------------------------------------------------------------------ reference
def expect(table, lens, stack, count, BLOCK, N, add=None, keep=None, starts=None):
    """(table, stack, new_lens, count, slots, positions, status) by a list of free blocks."""
    table, stack, status = table.copy(), stack.copy(), 0
    B, maxb = table.shape
    cap, pool = maxb * BLOCK, len(stack)
    n = np.clip(lens, 0, cap)
    k = n if keep is None else np.clip(keep, 0, n)
    a = np.full(B, N) if add is None else np.clip(add, 0, N)
    if (n != lens).any() or (keep is not None and (k != keep).any()) or (add is not None and (a != add).any()):
        status |= 2
    if not 0 <= count <= pool:
        status, count = status | 2, min(max(count, 0), pool)
    up = lambda x: -(-int(x) // BLOCK)  # noqa: E731
    free = list(stack[:count])
    for b in range(B):
        for i in range(up(k[b] + a[b]), up(n[b])):
            if len(free) < pool:
                free.append(table[b, i])
            else:
                status |= 2
    new = n.copy()
    slots, pos = np.full((B, N), -1), np.full((B, N), -1)
    asked, there = 0, len(free)
    for b in range(B):
        have, need = up(n[b]), up(k[b] + a[b])
        if need > maxb:
            status |= 2
            continue
        asked += max(need - have, 0)
        if need > have and asked > there:
            status |= 16
            continue
        for i in range(have, need):
            table[b, i] = free.pop()
            if not 0 <= table[b, i] < pool:
                status |= 1
        new[b] = k[b] + a[b]
        for j in range(a[b]):
            t = k[b] + j
            p = table[b, t // BLOCK]
            slots[b, j] = p * BLOCK + t % BLOCK if 0 <= p < pool else -1
            pos[b, j] = t if starts is None else starts[b] + j
    for i in range(count, len(free)):
        stack[i] = free[i]
    return table, stack, new, len(free), slots, pos, status


# ------------------------------------------------------------------ CPU: refusals
def call(pa, B=2, N=3, BLOCK=16, ptr=None, nopts=False, **o):
    vals = dict(max_blocks=8, num_blocks=32, add=None, keep=None, starts=None, positions=None, status=None)
    vals.update(o)
    p = [(i + 1) * A for i in range(7)]
    for i, x in (ptr or {}).items():
        p[i] = x
    p = [None if x is None else ctypes.c_void_p(x) for x in p]
    return pa.LIB.pa_plan_blocks(*p, B, N, BLOCK, None if nopts else ctypes.byref(pa.BlocksOpts(**vals)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(nopts=True), NULL), *[(dict(ptr={i: None}), NULL) for i in range(7)],
    (dict(B=-1), DIMS), (dict(N=-1), DIMS), (dict(BLOCK=0), DIMS), (dict(max_blocks=0), DIMS), (dict(num_blocks=0), DIMS),
    (dict(max_blocks=1 << 26), DIMS), (dict(num_blocks=1 << 27), DIMS), (dict(B=4096, max_blocks=1 << 20, BLOCK=8), DIMS),
    (dict(B=1 << 20, N=1 << 12), DIMS), (dict(ptr={6: 1 * A}), DIMS), (dict(ptr={4: 2 * A + 4}), DIMS), (dict(ptr={5: 4 * A}), DIMS),
    (dict(add=1 * A), DIMS), (dict(positions=7 * A + 8), DIMS), (dict(status=3 * A), DIMS),
    (dict(B=4097), UNSUP), (dict(N=65537), UNSUP),
    *[(dict(ptr={i: (i + 1) * A + 2}), ALIGN) for i in range(7)], (dict(keep=9 * A + 1), ALIGN), (dict(starts=9 * A + 3), ALIGN),
])
def test_refusals(pa, kw, code):
    assert call(pa, **kw) == code


# ------------------------------------------------------------------ GPU
def state(seed, lens, BLOCK, maxb, spare):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens)
    used = [-(-int(min(max(n, 0), maxb * BLOCK)) // BLOCK) for n in lens]
    pool = sum(used) + spare
    ids = rng.permutation(pool).astype(np.int64)
    table = rng.integers(-5, 0, (len(lens), maxb))  # behind a sequence's blocks anything may stand
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = ids[at: at + u]
        at += u
    stack = np.full(max(pool, 1), -7)
    stack[:spare] = ids[at:]
    return table, lens, stack, spare


def check(pa, table, lens, stack, count, BLOCK, N, again=True, **kw):
    want = expect(table, lens, stack, count, BLOCK, N, **kw)
    d = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    t, s, status = d(table), d(stack), d([0])
    plan = pa.BlockPlan(t, d(lens), s, d([count]), BLOCK=BLOCK, width=N, status=status,
                        **{k: d(v) for k, v in kw.items() if v is not None})
    for x in (plan.new_lens, plan.slots, plan.positions, plan.new_free_count):
        x.fill_(-99)
    for _ in range(2 if again else 1):  # the same call again gives the same
        plan.run()
        torch.cuda.synchronize()
        got = (t, s, plan.new_lens, plan.new_free_count, plan.slots, plan.positions)
        for name, g, w in zip(("table", "stack", "new_lens", "count", "slots", "positions"), got, want):
            np.testing.assert_array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1), err_msg=name)
        assert int(status) == want[6]


@pytest.mark.gpu
@pytest.mark.parametrize("BLOCK", [8, 16, 64, 3, 1])
def test_one_token_each(pa, BLOCK):
    lens = [0, 1, BLOCK - 1, BLOCK, BLOCK + 1, 5 * BLOCK, 37, 3 * BLOCK - 1]
    check(pa, *state(1, lens, BLOCK, 64, 9), BLOCK, 1)


@pytest.mark.gpu
def test_done_replaced_and_shortened(pa):
    lens = [40, 17, 64, 5, 33, 80, 16, 0]
    keep = [0, 17, 20, 5, 0, 79, 0, 0]
    add = [0, 1, 1, 30, 40, 0, 3, 12]
    for spare in (0, 1, 3, 20):
        check(pa, *state(2, lens, 16, 8, spare), 16, 40, add=add, keep=keep)
        check(pa, *state(2, lens, 16, 8, spare), 16, 40, add=add, keep=keep, starts=np.arange(8) * 1000 - 3)


@pytest.mark.gpu
def test_too_few_blocks_and_rows_too_long(pa):
    lens = [16, 16, 10, 64, 16, 16, 127]
    for spare in range(6):
        check(pa, *state(3, lens, 16, 8, spare), 16, 70, add=[1, 20, 2, 70, 33, 0, 1])


@pytest.mark.gpu
def test_nothing(pa):
    check(pa, np.zeros((0, 4), int), np.zeros(0, int), np.full(5, 3), 4, 16, 2)      # no sequence
    check(pa, *state(4, [40, 3], 16, 4, 2), 16, 0, keep=[0, 3])                          # only given back
    check(pa, *state(4, [40, 3], 16, 4, 2), 16, 5, add=[0, 0])


@pytest.mark.gpu
def test_values_out_of_range_are_clamped_and_reported(pa):
    table, lens, stack, count = state(5, [40, 3, 50], 16, 4, 6)
    check(pa, table, np.array([-2, 3, 5000]), stack, count, 16, 4, add=[2, 9, -1], keep=[3, 3, 60])
    check(pa, table, lens, stack, 10 ** 6, 16, 1, again=False)
    check(pa, table, lens, stack, -4, 16, 1)
    # blocks outside the pool on the stack
    stack[:6] = [10 ** 6, -3, 5, 2 ** 30, 1, 2]
    check(pa, table, lens, stack, count, 16, 30)
    # a stack that cannot hold what comes back
    check(pa, table, lens, stack[:7], 6, 16, 1, keep=[0, 0, 0], again=False)


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(6))
def test_drawn(pa, seed):
    rng = np.random.default_rng(seed)
    B = int(rng.choice([1, 3, 31, 500, 513, 1100, 4096]))
    BLOCK, N, maxb = int(rng.choice([8, 16, 32, 64])), int(rng.choice([1, 2, 17, 300])), int(rng.integers(6, 40))
    lens = rng.integers(0, maxb * BLOCK - min(N, 4 * BLOCK), B)
    keep = np.where(rng.random(B) < 0.2, 0, np.where(rng.random(B) < 0.3, lens // 2, lens))
    add = rng.integers(0, N + 1, B)
    check(pa, *state(seed, lens, BLOCK, maxb, int(rng.integers(0, B * (N // BLOCK + 1) + 1))), BLOCK, N, add=add, keep=keep)


@pytest.mark.gpu
def test_a_long_prompt_in_a_large_batch(pa):
    lens = np.arange(40) * 7 % 50
    add = np.where(np.arange(40) % 13 == 5, 65536, 1)
    check(pa, *state(7, lens, 64, 1040, 5000), 64, 65536, add=add)


@pytest.mark.gpu
def test_a_loop_gives_every_block_to_one_sequence(pa):
    """Steps with arrivals, ends and one eviction: at every step the blocks in
    use and the free ones are the pool, each once."""
    rng = np.random.default_rng(11)
    B, BLOCK, maxb, pool = 12, 8, 10, 70
    d = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    table, stack = d(np.full((B, maxb), -1)), d(rng.permutation(pool))
    lens, count, status = d(np.zeros(B)), d([pool]), d([0])
    keep, add = d(np.zeros(B)), d(np.zeros(B))
    plan = pa.BlockPlan(table, lens, stack, count, BLOCK=BLOCK, width=20, add=add, keep=keep, status=status)
    for step in range(40):
        n = lens.cpu().numpy()
        k = np.where(rng.random(B) < 0.1, 0, n)
        if step == 20:
            k = n // 2
        a = np.where(k == 0, rng.integers(0, 21, B), 1)
        keep.copy_(d(k)), add.copy_(d(a))
        new, left, slots, _ = plan.run()
        torch.cuda.synchronize()
        new, left = new.cpu().numpy(), int(left)
        used = np.concatenate([table[b, : -(-int(new[b]) // BLOCK)].cpu().numpy() for b in range(B)])
        everything = np.concatenate((used, stack[:left].cpu().numpy()))
        assert sorted(everything) == list(range(pool))
        lens.copy_(plan.new_lens), count.copy_(plan.new_free_count)


@pytest.mark.gpu
def test_refused_tensors(pa):
    d = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    good = dict(block_table=d([[0, 1], [2, 3]]), seq_lens=d([3, 4]), free_blocks=d([4, 5, 6, 7, 0, 0, 0, 0]), free_count=d([4]))
    pa.plan_blocks(**good, BLOCK=8, width=1)
    for name, bad in (("block_table", good["block_table"].long()), ("seq_lens", d([3])), ("free_count", d([1, 2])),
                      ("free_blocks", good["free_blocks"].view(2, 4)), ("seq_lens", torch.tensor([3, 4], dtype=torch.int32)),
                      ("block_table", d([[0, 1, 1], [2, 3, 3]])[:, :2])):
        with pytest.raises(ValueError):
            pa.plan_blocks(**{**good, name: bad}, BLOCK=8, width=1)
    for kw in (dict(BLOCK=8, width=-1), dict(BLOCK=2 ** 32 + 8, width=1), dict(BLOCK=8, width=2 ** 32)):
        with pytest.raises(ValueError):
            pa.plan_blocks(**good, **kw)
    with pytest.raises(pa.PagedAttentionError):
        pa.plan_blocks(**good, BLOCK=0, width=1)
