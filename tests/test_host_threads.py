"""Calls of one kernel from several host threads at once, each on a stream of its own."""
import threading

import numpy as np
import pytest
import torch

from test_q8 import Cache, ints, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_182_gb300 import binding

    return binding


def _decode(pa, B, seed):
    c = Cache(seed, [33] * B, 1, 64, 16)
    return pa.Q8Plan(rows_of(c.rng, "f16", B, 2, 1, 64).cuda(), *c.cuda(), ints(c.lens), scale=0.125)


def _select(pa, maxb, seed):
    c = Cache(seed, [200], 1, 64, 16, width=8)
    dev = c.cuda()
    table = ints(c.rng.integers(0, len(c.ks), (1, maxb)))
    return pa.Q8SelectPlan(rows_of(c.rng, "f16", 1, 2, 1, 64).cuda(), torch.from_numpy(c.bounds).cuda(), dev[2], table,
                           ints([maxb * 16 - 5]), BLOCK=16, budget=9)


def _blocks(pa, B, seed):
    return pa.BlockPlan(ints(np.arange(2 * B).reshape(B, 2)), ints([16] * B), ints(np.arange(2 * B)), ints([0]), BLOCK=16, width=1)


def _gradient(pa, D, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    q, k, v, y, go = (torch.randn(1, 2, 40, D, generator=g, device="cuda") for _ in range(5))
    return pa.VjpPlan(q, k, v, y, go, scale=0.1, causal=True)


def _evict(pa, D, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    kc, vc = (torch.randn(8, 16, 100, D, generator=g, device="cuda") for _ in range(2))
    return pa.EvictPlan(kc, vc, ints([[0, 1, 2]]), ints([40]), torch.rand(1, 48, generator=g, device="cuda"), budget=20,
                        dst_table=ints([[4, 5]]))


@pytest.mark.parametrize("make,sizes", [(_decode, (3, 70)), (_select, (2500, 20000)), (_blocks, (2200, 4096)),
                                        (_gradient, (64, 256)), (_evict, (128, 160))])
def test_two_host_threads_at_once(pa, make, sizes):
    """Calls of one kernel that need unlike amounts of shared memory, each on a stream of its own."""
    plans = [make(pa, n, i) for i, n in enumerate(sizes)]
    torch.cuda.synchronize()
    streams, failed, go = [torch.cuda.Stream() for _ in plans], [], threading.Barrier(2)

    def work(plan, stream):
        go.wait()
        try:
            for _ in range(3000):
                plan.run(stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=x) for x in zip(plans, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
