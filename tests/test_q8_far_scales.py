"""Attention over a cache in 8 bits whose value scales lie far apart."""
import math

import numpy as np
import pytest
import torch

from test_q8 import DT, Cache, as64, attend, ints, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_182_gb300 import binding

    return binding


# value scales of whole blocks; their keys all weigh much the same, or one block's most of all
FAR = [(2.0 ** -96, 2.0 ** 60), (2.0 ** -96, 2.0 ** 90), (2.0 ** -96, 1.0), (2.0 ** -40, 2.0 ** 70), (2.0 ** -31, 2.0 ** 31), (2.0 ** -33, 2.0 ** 33)]


@pytest.mark.parametrize("fmt", ["f32", "bf16"])
@pytest.mark.parametrize("B,KV,G,NQ,D,BLOCK,n", [(1, 2, 4, 1, 128, 16, 700), (1, 1, 3, 1, 64, 8, 9000), (2, 1, 16, 1, 128, 32, 900),
                                                 (3, 1, 8, 4, 64, 8, 3000), (700, 1, 2, 1, 64, 16, 130), (160, 2, 1, 1, 128, 64, 500)])
def test_value_scales_far_apart(pa, fmt, B, KV, G, NQ, D, BLOCK, n):
    """A key's share in the softmax does not depend on the size of its value, nor on who joins it with the others."""
    for near, far in FAR:
        c = Cache(61, [n] * B, KV, D, BLOCK)
        c.lens = np.maximum(c.lens - np.arange(B) % 37, 1).astype(np.int32)
        few = c.rng.random(c.vs.shape)
        q = rows_of(c.rng, fmt, B, KV * G, NQ, D)
        for share, weigh in ((0.5, 0.0), (0.02, 0.0), (0.95, 0.0), (0.05, 0.5)):
            c.vs = np.where(few < share, np.float32(far), np.float32(near))
            x = q * (0.2 + weigh)
            attend(pa, c, x, fmt, True) if B < 10 else few_of(pa, c, x, fmt)


def few_of(pa, c, q, fmt):
    """As `attend`, of a large batch a few sequences compared."""
    scale = float(np.float32(c.D ** -0.5))
    out = pa.decode_q8(q.cuda(), *c.cuda(), ints(c.lens), scale=scale, causal=True)
    torch.cuda.synchronize()
    lens, table = c.lens, c.table
    for b in (0, 1, len(lens) // 2, len(lens) - 1):
        c.lens, c.table = lens[b: b + 1], table[b: b + 1]
        want, tol = c.attend(as64(q[b: b + 1]), scale, True, fmt)
        assert np.all(np.abs(as64(out[b: b + 1]) - want) <= tol), b
    c.lens, c.table = lens, table


def test_one_block_of_zeros_beside_large_values(pa):
    """Equal scores: the output is the large block's value times its share of the keys, exactly known."""
    for fmt in ("f32", "bf16"):
        for far in (2.0 ** 50, 2.0 ** 96):
            c = Cache(62, [64], 1, 64, 16)
            c.vs[:] = np.float32(2.0 ** -96)
            c.vs[c.table[0, 1]] = np.float32(far)
            c.vc[:] = 0
            c.vc[c.table[0, 1]] = 100
            out = pa.decode_q8(torch.zeros(1, 4, 1, 64, dtype=DT[fmt], device="cuda"), *c.cuda(), ints(c.lens), scale=0.125)
            torch.cuda.synchronize()
            np.testing.assert_allclose(as64(out), 25 * far, rtol=2.0 ** -7, atol=0)


def test_bits_do_not_depend_on_blocks_of_others(pa):
    """Scales of blocks that no sequence has, the pool's first among them, change no bit."""
    c = Cache(63, [100, 61], 2, 64, 8, spare=3)
    own = c.table.reshape(-1)
    free = [p for p in range(len(c.ks)) if p not in own]
    if 0 in own:  # block 0 to nobody
        c.table[c.table == 0] = free[0]
        free[0] = 0
    q = rows_of(c.rng, "f16", 2, 4, 1, 64).cuda()
    got = []
    for vs, ks in ((1.0, 1.0), (0.0, 0.0), (2.0 ** 100, 2.0 ** 100), (math.inf, math.nan), (math.nan, math.inf)):
        c.vs[free], c.ks[free] = np.float32(vs), np.float32(ks)
        got.append(pa.decode_q8(q, *c.cuda(), ints(c.lens), scale=0.125))
    torch.cuda.synchronize()
    for x in got[1:]:
        assert torch.equal(x, got[0])


@pytest.mark.parametrize("G,NQ", [(2, 1), (12, 1), (8, 4)])
@pytest.mark.parametrize("near,far", [(2.0 ** -96, 4.0), (0.0, 2.0 ** -10), (2.0 ** -60, 1.0)])
def test_float16_outputs_beside_small_value_scales(pa, G, NQ, near, far):
    """Zeros and near zeros beside ordinary values, as a padded cache has them."""
    for B, n, D, BLOCK in ((1, 12000, 64, 8), (2, 500, 128, 16)):
        c = Cache(64, [n] * B, 1, D, BLOCK)
        for share in (0.1, 0.9):
            c.vs = np.where(c.rng.random(c.vs.shape) < share, np.float32(far), np.float32(near)).astype(np.float32)
            attend(pa, c, rows_of(c.rng, "f16", B, G, NQ, D) * 0.5, "f16", True)
