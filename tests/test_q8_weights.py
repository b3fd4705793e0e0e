"""Attention over a cache in 8 bits: a weight's digits, seen where values cancel.

Tokens come in pairs of opposite values and nearly equal weights: the output is a small
difference, and what a weight loses in its rounding stands out against the output's own
rounding, which is relative to that difference.  With value scales of one and small
scores the bound of `test_q8` (its docstring), without its weight of 11 bits, is about
2^-15 of sum p |v|; weights of 11 bits alone are off by up to 2^-11 of it."""
import math

import numpy as np
import pytest
import torch

from test_q8 import Cache, as64, ints, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_182_gb300 import binding

    return binding


def bound(c, q, scale, fmt):
    """(outputs, bounds of their errors) of non-causal attention in 64 bits."""
    B, H, NQ, D = q.shape
    G = H // c.KV
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    half = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[fmt]
    digits, sums = (2.0 ** -22, 2.0 ** -20) if fmt == "f32" else (2.0 ** -36, 2.0 ** -16)
    for b, n in enumerate(c.lens.tolist()):
        for h in range(c.KV):
            K, V = c.rows(b, np.arange(n), h)
            x = q[b, h * G: (h + 1) * G].reshape(-1, D)
            s = scale * (x @ K.T)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            mag = scale * math.log2(math.e) * (np.abs(x) @ np.abs(K).T * D * 2.0 ** -23 + digits * np.abs(x).max(1)[:, None] * np.abs(K).sum(1))
            t = np.abs(s) * math.log2(math.e)
            e = 2 * math.log(2) * (mag + 2.0 ** -20 * (1 + t + t.max(1, keepdims=True))).max(1)
            y = p @ V
            out[b, h * G: (h + 1) * G] = y.reshape(G, NQ, D)
            tol[b, h * G: (h + 1) * G] = ((e + 2.0 ** -22 + sums)[:, None] * (p @ np.abs(V)) + n * 2.0 ** -31 * np.abs(V).max()
                                          + half * np.abs(y) + (2.0 ** -25 if fmt == "f16" else 0)).reshape(G, NQ, D)
    return out, tol


@pytest.mark.parametrize("fmt,G,NQ", [("f16", 1, 1), ("f16", 4, 2), ("f16", 12, 1), ("f16", 8, 4), ("f16", 20, 3), ("bf16", 1, 1), ("bf16", 8, 1),
                                      ("f32", 4, 1), ("f32", 8, 3)])
@pytest.mark.parametrize("D,BLOCK,B,n", [(128, 16, 3, 6), (64, 8, 5, 40), (64, 32, 400, 10), (128, 64, 1, 6000)])
def test_weights_keep_their_digits(pa, fmt, G, NQ, D, BLOCK, B, n):
    c = Cache(70, [n] * B, 1, D, BLOCK)
    c.lens = np.maximum(c.lens - np.arange(B) % 3 * 2, 2).astype(np.int32)  # (even: whole pairs)
    c.vs[:] = 1
    c.vc[:, 1::2] = -c.vc[:, ::2]
    q = rows_of(c.rng, fmt, B, G, NQ, D) * 0.125
    scale = 2.0 ** -4
    out = pa.decode_q8(q.cuda(), *c.cuda(), ints(c.lens), scale=scale)
    torch.cuda.synchronize()
    want, tol = bound(c, as64(q), scale, fmt)
    off = np.abs(as64(out) - want)
    assert np.all(off <= tol), f"{(off / tol).max()} of the bound"
