"""Attention over a cache in 8 bits: lengths out of range beside selected lists."""
import numpy as np
import pytest
import torch

from test_q8 import Cache, as64, attend, ints, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_182_gb300 import binding

    return binding


def test_a_length_out_of_range_beside_selected_blocks(pa):
    """Clamped and reported as without the lists, in each way of dealing the work."""
    for B in (2, 60, 700):
        c = Cache(60, [40] * B, 1, 64, 16)
        q = rows_of(c.rng, "f16", B, 2, 1, 64)
        sel, cnt = np.tile(np.array([0, 2], np.int32), (B, 1, 1)), np.full((B, 1), 2)
        attend(pa, c, q, "f16", False, selected=sel, counts=cnt)
        for n, seen in ((49, 48), (2 ** 31 - 1, 48), (-1, 0)):
            lens, st = c.lens.copy(), ints([0])
            lens[B - 1] = n
            if n < 0:
                sel[B - 1] = -1
            out = pa.decode_q8(q.cuda(), *c.cuda(), ints(lens), scale=0.125, selected=ints(sel), counts=ints(cnt), status=st)
            torch.cuda.synchronize()
            assert int(st) == 2, (B, n)
            keep, c.lens = c.lens, c.lens.copy()
            c.lens[B - 1] = seen
            want, tol = c.attend(as64(q), 0.125, False, "f16", sel, cnt)
            assert np.all(np.abs(as64(out) - want) <= tol)
            c.lens = keep
