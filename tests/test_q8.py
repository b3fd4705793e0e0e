"""The cache in 8 bits (include/pa_q8.h): refusals on the CPU; on the GPU the
store, the read, the selection and the attention against plain 64-bit
arithmetic.

Codes, scales, bounds and selections are whole numbers or are rounded once by
their definition, so they are compared exactly.  A read is one rounding of a
float32 product (the test does the same in numpy, exactly).

Bound of an attention output (row with weights p, t = log2(e) scale q.k):
  * scores: the product of the codes with q's digits is exact, its sum of D
    terms in float32 off by at most D 2^-23 of sum |q k|; digits of q below
    2^-22 of the row's largest (float32: two fp16 parts) are lost: 2^-22 |q|max
    sum |k|; the scale's products, the sum with log2(v_scale), the maximum's
    difference, log2 and exp2 come to 2^-20 (1 + |t| + |log2 v_scale|) in t;
  * weights: rounded to fp16, at most 2^-11 of each (half a step; float32: two
    parts, 2^-22), or 2^-25 absolutely, where the row's largest is at least
    2^6: 2^-31 of it;
  * sums in float32 over n terms and the joins of at most 304 pieces: 2^-16
    for the tensor cores' sums (n / 16 / 8 steps of a warp at 2^-23 each for n
    up to 16384), 2^-20 where float32 sums are rounded additions;
  * the output's own rounding: half a step of its type.
With e the relative error of a weight (2 ln 2 times the score's, for weight and
sum), |error| <= (e + weight + sums) sum p |v| + n 2^-31 max |v| + half a step.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
A = 1 << 24
NULL, DIMS, UNSUP, ALIGN, WORK = -1, -2, -3, -4, -5
SMALLEST = 2.0 ** -96


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_182_gb300 import _build

    _build.build()
    from paged_kv_cache_182_gb300 import binding

    return binding


# ------------------------------------------------------------------ CPU: refusals
def pointers(n, ptr):
    p = [(i + 1) * A for i in range(n)]
    for i, x in (ptr or {}).items():
        p[i] = x
    return [None if x is None else ctypes.c_void_p(x) for x in p]


def append(pa, B=2, KV=2, D=64, N=3, BLOCK=16, ptr=None, nopts=False, ks=(384, 192, 64), vs=(384, 192, 64), **o):
    opts = pa.Q8AppendOpts(**{**dict(max_blocks=8, num_blocks=32, dtype=1, counts=None, bounds=None, status=None), **o})
    opts.k_strides[:], opts.v_strides[:] = ks, vs
    return pa.LIB.pa_q8_append(*pointers(8, ptr), B, KV, D, N, BLOCK, None if nopts else ctypes.byref(opts), None)


def read(pa, B=2, KV=2, D=64, N=3, BLOCK=16, ptr=None, nopts=False, **o):
    opts = pa.Q8ReadOpts(**{**dict(max_blocks=8, num_blocks=32, dtype=1, counts=None, status=None), **o})
    return pa.LIB.pa_q8_read(*pointers(8, ptr), B, KV, D, N, BLOCK, None if nopts else ctypes.byref(opts), None)


def select(pa, B=2, H=4, KV=2, D=64, NQ=1, BLOCK=16, ptr=None, nopts=False, **o):
    opts = pa.Q8SelectOpts(**{**dict(max_blocks=8, num_blocks=32, dtype=1, budget=4, keep_first=1, keep_last=1, status=None), **o})
    return pa.LIB.pa_q8_select(*pointers(7, ptr), B, H, KV, D, NQ, BLOCK, None if nopts else ctypes.byref(opts), None)


def decode(pa, B=2, H=4, KV=2, D=64, NQ=1, BLOCK=16, ptr=None, nopts=False, **o):
    opts = pa.Q8Opts(**{**dict(max_blocks=8, num_blocks=32, dtype=1, causal=1, selected=None, counts=None, budget=0,
                               workspace=20 * A, workspace_bytes=1 << 30, status=None), **o})
    return pa.LIB.pa_q8_decode(*pointers(8, ptr), ctypes.c_float(0.1), B, H, KV, D, NQ, BLOCK, None if nopts else ctypes.byref(opts), None)


COMMON = [(dict(nopts=True), NULL), (dict(B=-1), DIMS), (dict(KV=0), DIMS), (dict(D=0), DIMS), (dict(max_blocks=0), DIMS),
          (dict(num_blocks=0), DIMS), (dict(max_blocks=1 << 26), DIMS), (dict(num_blocks=1 << 27), DIMS), (dict(D=80), UNSUP),
          (dict(D=256), UNSUP), (dict(BLOCK=24), UNSUP), (dict(BLOCK=128), UNSUP), (dict(dtype=3), UNSUP), (dict(dtype=-1), UNSUP),
          (dict(B=4097), UNSUP), (dict(status=16 * A + 2), ALIGN)]


@pytest.mark.parametrize("kw,code", COMMON + [
    *[(dict(ptr={i: None}), NULL) for i in range(8)], (dict(N=-1), DIMS), (dict(N=65537), UNSUP), (dict(KV=1025), UNSUP),
    (dict(ks=(-8, 0, 0)), ALIGN), (dict(vs=(384, 4, 64)), ALIGN), (dict(ptr={4: 5 * A + 8}), ALIGN), (dict(ptr={0: A + 8}), ALIGN),
    (dict(ptr={2: 3 * A + 2}), ALIGN), (dict(bounds=12 * A + 4), ALIGN), (dict(counts=12 * A + 1), ALIGN),
    (dict(ptr={1: 1 * A}), DIMS), (dict(ptr={5: 2 * A + 64}), DIMS), (dict(ptr={3: 3 * A + 8}), DIMS), (dict(bounds=1 * A), DIMS),
    (dict(ptr={7: 4 * A}), DIMS), (dict(counts=12 * A, bounds=12 * A), DIMS), (dict(ks=(1 << 41, 8, 8)), DIMS),
])
def test_append_refusals(pa, kw, code):
    assert append(pa, **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    *[(dict(ptr={i: None}), NULL) for i in range(8)], (dict(N=-1), DIMS), (dict(N=1 << 30), DIMS),
    (dict(ptr={6: 7 * A + 8}), ALIGN), (dict(ptr={5: 6 * A + 1}), ALIGN), (dict(ptr={7: 7 * A}), DIMS), (dict(ptr={6: 1 * A}), DIMS),
    (dict(ptr={6: 5 * A}), DIMS), (dict(counts=7 * A), DIMS),
])
def test_read_refusals(pa, kw, code):
    assert read(pa, **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    *[(dict(ptr={i: None}), NULL) for i in range(7)], (dict(H=0), DIMS), (dict(H=5), DIMS), (dict(NQ=0), DIMS), (dict(NQ=17), UNSUP),
    (dict(H=256, KV=2, NQ=16), UNSUP), (dict(budget=0), DIMS), (dict(budget=1 << 30), DIMS), (dict(keep_first=-1), DIMS),
    (dict(keep_last=-1), DIMS), (dict(keep_first=2, keep_last=3), DIMS), (dict(max_blocks=32769), UNSUP),
    (dict(B=4096, KV=16, H=16), UNSUP), (dict(ptr={0: A + 4}), ALIGN), (dict(ptr={1: 2 * A + 8}), ALIGN), (dict(ptr={6: 7 * A + 2}), ALIGN),
    (dict(ptr={6: 6 * A}), DIMS), (dict(ptr={5: 4 * A}), DIMS),
])
def test_select_refusals(pa, kw, code):
    assert select(pa, **kw) == code


@pytest.mark.parametrize("kw,code", COMMON + [
    *[(dict(ptr={i: None}), NULL) for i in range(8)], (dict(H=0), DIMS), (dict(H=5), DIMS), (dict(NQ=0), DIMS), (dict(NQ=17), UNSUP),
    (dict(H=256, KV=2, NQ=16), UNSUP), (dict(selected=12 * A), NULL), (dict(counts=12 * A), NULL),
    (dict(selected=12 * A, counts=13 * A, budget=0), DIMS), (dict(selected=12 * A, counts=13 * A, budget=1 << 26), DIMS),
    (dict(selected=12 * A, counts=13 * A, budget=2, B=4096, KV=4), UNSUP), (dict(ptr={7: 8 * A + 8}), ALIGN),
    (dict(workspace=None), WORK), (dict(workspace_bytes=1000), WORK), (dict(workspace=20 * A + 128), WORK),
    (dict(ptr={7: 1 * A}), DIMS), (dict(ptr={7: 20 * A + 256}), DIMS), (dict(workspace=2 * A), DIMS),
])
def test_decode_refusals(pa, kw, code):
    assert decode(pa, **kw) == code


def test_nothing_to_do(pa):
    assert append(pa, B=0) == 0 and append(pa, N=0) == 0 and read(pa, B=0) == 0 and read(pa, N=0) == 0
    assert select(pa, B=0) == 0 and decode(pa, B=0) == 0


def test_workspace_sizes(pa):
    for f in (pa.q8_workspace_bytes, pa.q8_workspace_zero_bytes):
        assert f(0, 4, 2, 64, 1) == 0 and f(1, 5, 2, 64, 1) == 0 and f(1, 4, 2, 80, 1) == 0 and f(1, 4, 2, 64, 17) == 0
    assert pa.q8_workspace_bytes(4, 32, 8, 128, 4) > pa.q8_workspace_zero_bytes(4, 32, 8, 128, 4) >= 4 * 8 * 2 * 4


# ------------------------------------------------------------------ plain forms
def scale_of(x):
    fine = np.abs(x[np.isfinite(x)])
    a = np.float32(fine.max()) / np.float32(127) if fine.size else np.float32(0)
    return max(np.float32(a), np.float32(SMALLEST))


def codes_of(x, scale):
    with np.errstate(invalid="ignore"):
        c = np.clip(np.rint(np.asarray(x, np.float64) / np.float64(scale)), -127, 127)
    return np.where(np.isnan(x), 0, c).astype(np.int8)


class Cache:
    """A cache in 8 bits on the host, as numpy."""

    def __init__(self, seed, lens, KV, D, BLOCK, more=0, spare=2, width=None):
        rng = np.random.default_rng(seed)
        self.rng, self.BLOCK, self.KV, self.D, self.lens = rng, BLOCK, KV, D, np.asarray(lens, np.int32)
        maxb = width or max(1, max(-(-(int(n) + more) // BLOCK) for n in lens))
        pool = len(lens) * maxb + spare
        self.table = rng.permutation(pool)[: len(lens) * maxb].reshape(len(lens), maxb).astype(np.int32)
        self.kc, self.vc = (rng.integers(-127, 128, (pool, BLOCK, KV, D)).astype(np.int8) for _ in range(2))
        self.ks, self.vs = (np.exp(rng.normal(-4, 0.5, (pool, KV))).astype(np.float32) for _ in range(2))
        self.bounds = np.stack((self.kc.min(1), self.kc.max(1)), 2)

    def slot(self, b, i):
        return int(self.table[b, i // self.BLOCK]), i % self.BLOCK

    def append(self, kn, vn, counts, bounds):
        for b, n in enumerate(self.lens.tolist()):
            m = int(counts[b])
            for i in range(n // self.BLOCK, -(-(n + m) // self.BLOCK) if m else 0):
                p, a, z = int(self.table[b, i]), max(n, i * self.BLOCK), min(n + m, (i + 1) * self.BLOCK)
                old = a - i * self.BLOCK
                for h in range(self.KV):
                    for cache, scale, new in ((self.kc, self.ks, kn), (self.vc, self.vs, vn)):
                        rows = new[b, h, a - n: z - n]
                        was = scale[p, h] if old else np.float32(0)
                        now = max(scale_of(rows), was)
                        c = codes_of(rows, now)
                        if now > was and old:
                            cache[p, :old, h] = codes_of(cache[p, :old, h].astype(np.float64) * np.float64(was), now)
                        cache[p, old: old + len(c), h] = c
                        scale[p, h] = now
                        if cache is self.kc and bounds:
                            every = cache[p, : old + len(c), h]
                            self.bounds[p, h] = every.min(0), every.max(0)

    def rows(self, b, ids, h):
        p, r = self.table[b, ids // self.BLOCK], ids % self.BLOCK
        return tuple(c[p, r, h].astype(np.float64) * np.maximum(s[p, h], SMALLEST).astype(np.float64)[:, None]
                     for c, s in ((self.kc, self.ks), (self.vc, self.vs)))

    def select(self, q, budget, first, last):
        B, H, NQ, D = q.shape
        G = H // self.KV
        sel, cnt = np.full((B, self.KV, budget), -1, np.int32), np.zeros((B, self.KV), np.int32)
        for b in range(B):
            nb = -(-int(self.lens[b]) // self.BLOCK)
            for h in range(self.KV):
                ids = np.arange(nb)
                if nb > budget:
                    score = np.full(nb, -np.inf, np.float32)
                    p = self.table[b, :nb]
                    ends = self.bounds[p, h].astype(np.int64)
                    for row in q[b, h * G: (h + 1) * G].reshape(-1, D):
                        qs = scale_of(row)
                        c = codes_of(row, qs).astype(np.int64)
                        total = np.maximum(c * ends[:, 0], c * ends[:, 1]).sum(1)
                        with np.errstate(over="ignore", invalid="ignore"):
                            score = np.fmax(score, (qs * self.ks[p, h]) * total.astype(np.float32))
                    mid = np.arange(first, nb - last)
                    best = mid[np.lexsort((mid, -score[mid]))][: budget - first - last]
                    ids = np.sort(np.concatenate((np.arange(first), best, np.arange(nb - last, nb))))
                sel[b, h, : len(ids)], cnt[b, h] = ids, len(ids)
        return sel, cnt

    def attend(self, q, scale, causal, fmt, selected=None, counts=None):
        """(outputs, bounds of their errors) in 64 bits."""
        B, H, NQ, D = q.shape
        G = H // self.KV
        out, tol = np.zeros(q.shape), np.zeros(q.shape)
        digits = 2.0 ** -22 if fmt == "f32" else 2.0 ** -36
        weight, sums = (2.0 ** -22, 2.0 ** -20) if fmt == "f32" else (2.0 ** -11, 2.0 ** -16)
        half = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[fmt]
        for b, n in enumerate(self.lens.tolist()):
            for h in range(self.KV):
                ids = np.arange(n)
                if selected is not None:
                    own = selected[b, h, : counts[b, h]]
                    own = own[(own >= 0) & (own < -(-n // self.BLOCK))]
                    ids = (own[:, None] * self.BLOCK + np.arange(self.BLOCK)).reshape(-1)
                    ids = ids[ids < n]
                if not len(ids):
                    continue
                K, V = self.rows(b, ids, h)
                lv = np.abs(np.log2(np.maximum(self.vs[self.table[b, ids // self.BLOCK], h], SMALLEST)))
                for g in range(G):
                    for r in range(NQ):
                        x = q[b, h * G + g, r].astype(np.float64)
                        seen = ids <= n - NQ + r if causal else np.ones(len(ids), bool)
                        if not seen.any():
                            continue
                        k, v = K[seen], V[seen]
                        s = scale * (k @ x)
                        p = np.exp(s - s.max())
                        p /= p.sum()
                        y = p @ v
                        mag = scale * math.log2(math.e) * (np.abs(k) @ np.abs(x) * D * 2.0 ** -23
                                                           + digits * np.abs(x).max() * np.abs(k).sum(1))
                        t = np.abs(s) * math.log2(math.e)
                        e = 2 * math.log(2) * (mag + 2.0 ** -20 * (1 + t + t.max() + 2 * lv[seen])).max()
                        out[b, h * G + g, r] = y
                        tol[b, h * G + g, r] = ((e + weight + sums) * (p @ np.abs(v)) + len(k) * 2.0 ** -31 * np.abs(v).max()
                                                + half * np.abs(y) + (2.0 ** -25 if fmt == "f16" else 0))
        return out, tol

    def cuda(self):
        d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        return d(self.kc), d(self.vc), d(self.ks), d(self.vs), d(self.table)


def rows_of(rng, fmt, *shape):
    return torch.from_numpy(rng.normal(0, 1, shape).astype(np.float32)).to(DT[fmt])


def as64(t):
    return t.detach().cpu().double().numpy()


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ GPU: store
def store(pa, c, kn, vn, counts=None, bounds=True, status=None, want_status=0):
    """Both the kernel's store and the plain one of new rows (on the host), compared; the device's cache."""
    dev = c.cuda()
    db = torch.from_numpy(c.bounds.copy()).cuda()
    st = ints([0])
    got = pa.cache_append_q8(kn.cuda(), vn.cuda(), *dev, ints(c.lens), counts=None if counts is None else ints(counts),
                             bounds=db if bounds else None, status=st)
    torch.cuda.synchronize()
    assert int(st) == want_status
    n = kn.shape[2]
    c.append(kn.float().numpy(), vn.float().numpy(), [n] * len(c.lens) if counts is None else counts, bounds)
    for name, g, w in zip(("k_cache", "v_cache", "k_scale", "v_scale"), got, (c.kc, c.vc, c.ks, c.vs)):
        np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)
    np.testing.assert_array_equal(db.cpu().numpy(), c.bounds)
    return dev, db


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,BLOCK,KV", [(64, 8, 3), (64, 16, 1), (64, 32, 5), (64, 64, 2), (128, 8, 1), (128, 16, 3), (128, 32, 2), (128, 64, 1)])
def test_append(pa, fmt, D, BLOCK, KV):
    lens = [0, 1, BLOCK - 1, BLOCK, 2 * BLOCK + 3, 5]
    for N in (1, 2, BLOCK, 2 * BLOCK + 5):
        c = Cache(N, lens, KV, D, BLOCK, more=N)
        kn, vn = (rows_of(c.rng, fmt, len(lens), KV, N, D) * s for s in (0.7, 3))
        store(pa, c, kn, vn)
        c = Cache(N + 100, lens, KV, D, BLOCK, more=N)
        kn, vn = (rows_of(c.rng, fmt, len(lens), KV, N, D) * 10.0 ** e for e in (-4, 4))
        store(pa, c, kn, vn, counts=[N, 0, 1, max(0, N - 1), N, N // 2], bounds=N == 2)


@pytest.mark.gpu
def test_append_token_by_token_and_halves(pa):
    """Every step of a block's growth, values that lie on or next to half a step."""
    c = Cache(3, [0, 6], 2, 64, 16, more=40)
    dev, db = c.cuda(), torch.from_numpy(c.bounds.copy()).cuda()
    lens = ints(c.lens)
    for step in range(40):
        kn = torch.from_numpy((c.rng.integers(-254, 255, (2, 2, 1, 64)) / 2).astype(np.float32)) * (1 + step % 5)
        kn[..., 0] = 127 * (1 + step % 5)
        vn = torch.nextafter(kn, kn * 2)
        pa.cache_append_q8(kn.cuda(), vn.cuda(), *dev, lens, bounds=db)
        c.append(kn.numpy(), vn.numpy(), [1, 1], True)
        c.lens = c.lens + 1
        lens += 1
        torch.cuda.synchronize()
        for g, w in zip(dev, (c.kc, c.vc, c.ks, c.vs)):
            np.testing.assert_array_equal(g.cpu().numpy(), w)
        np.testing.assert_array_equal(db.cpu().numpy(), c.bounds)


@pytest.mark.gpu
def test_append_of_what_is_not_finite_and_of_zeros(pa):
    for fmt in DT:
        c = Cache(4, [3, 16, 0], 1, 64, 16, more=4)
        kn, vn = (rows_of(c.rng, fmt, 3, 1, 4, 64) for _ in range(2))
        kn[0, 0, 0, 3], kn[0, 0, 1, 5], kn[1, 0, 0, 0] = math.inf, -math.inf, math.nan
        vn[1] = math.nan
        vn[2] = 0
        kn[2] = 1e-40 if fmt != "f16" else 0  # below the least scale
        store(pa, c, kn, vn, want_status=32)


@pytest.mark.gpu
def test_append_strided_rows(pa):
    for fmt in DT:
        c = Cache(5, [0, 20], 3, 128, 16, more=9)
        both = rows_of(c.rng, fmt, 2, 9, 8, 128).cuda()
        kn, vn = both[:, :, 1:4].transpose(1, 2), both[:, :, 5:].transpose(1, 2)
        dev = c.cuda()
        pa.cache_append_q8(kn, vn, *dev, ints(c.lens))
        torch.cuda.synchronize()
        c.append(kn.float().cpu().numpy(), vn.float().cpu().numpy(), [9, 9], False)
        for g, w in zip(dev, (c.kc, c.vc, c.ks, c.vs)):
            np.testing.assert_array_equal(g.cpu().numpy(), w)


@pytest.mark.gpu
def test_append_without_a_block(pa):
    """Rows beyond the table or with an entry outside the pool: not stored, reported, the others as ever."""
    c = Cache(6, [14, 30, 5], 2, 64, 16, more=0, width=2)
    c.table[2, 0] = 10 ** 6
    keep = [x.copy() for x in (c.kc, c.vc, c.ks, c.vs)]
    dev, st = c.cuda(), ints([0])
    kn, vn = (rows_of(c.rng, "f16", 3, 2, 4, 64) for _ in range(2))
    pa.cache_append_q8(kn.cuda(), vn.cuda(), *dev, ints(c.lens), status=st)
    torch.cuda.synchronize()
    assert int(st) == 8
    c.append(kn.float().numpy(), vn.float().numpy(), [4, 2, 0], False)
    for g, w, k in zip(dev, (c.kc, c.vc, c.ks, c.vs), keep):
        np.testing.assert_array_equal(g.cpu().numpy(), w)
    # lengths out of range: clamped and reported
    st.zero_()
    pa.cache_append_q8(kn.cuda(), vn.cuda(), *dev, ints([-1, 1000, 0]), counts=ints([0, 9, -4]), status=st)
    torch.cuda.synchronize()
    assert int(st) == 2 + 8


@pytest.mark.gpu
def test_append_behind_4_gib(pa):
    """Blocks whose codes begin behind 2^32 bytes."""
    KV, D, BLOCK, pool = 8, 128, 64, 66000  # 4.3 GB of keys
    kc, vc = (torch.zeros(pool, BLOCK, KV, D, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(pool, KV, device="cuda") for _ in range(2))
    c = Cache(7, [70, 3], KV, D, BLOCK, more=5)
    far = c.table + pool - c.table.max() - 1
    for b in range(2):
        for i in range(c.table.shape[1]):
            for x, y in ((kc, c.kc), (vc, c.vc), (ks, c.ks), (vs, c.vs)):
                x[int(far[b, i])] = torch.from_numpy(y[c.table[b, i]])
    kn, vn = (rows_of(c.rng, "bf16", 2, KV, 5, D) for _ in range(2))
    pa.cache_append_q8(kn.cuda(), vn.cuda(), kc, vc, ks, vs, ints(far), ints(c.lens))
    c.append(kn.float().numpy(), vn.float().numpy(), [5, 5], False)
    c.lens = c.lens + 5
    ko, vo = pa.cache_read_q8(kc, vc, ks, vs, ints(far), ints([0, 0]), width=75, counts=ints(c.lens), dtype=torch.float32)
    q = rows_of(c.rng, "bf16", 2, 16, 1, D)
    out = pa.decode_q8(q.cuda(), kc, vc, ks, vs, ints(far), ints(c.lens), scale=0.09)
    torch.cuda.synchronize()
    for b, n in enumerate(c.lens.tolist()):
        for h in range(KV):
            K, V = c.rows(b, np.arange(n), h)
            np.testing.assert_array_equal(ko[b, h, :n].cpu().numpy(), K.astype(np.float32))
            np.testing.assert_array_equal(vo[b, h, :n].cpu().numpy(), V.astype(np.float32))
    want, tol = c.attend(q.double().numpy(), float(np.float32(0.09)), False, "bf16")
    assert np.all(np.abs(as64(out) - want) <= tol)


# ------------------------------------------------------------------ GPU: read
@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,BLOCK,KV", [(64, 8, 3), (128, 16, 1), (64, 64, 2), (128, 32, 8)])
def test_read(pa, fmt, D, BLOCK, KV):
    lens = [0, 1, 100, 3 * BLOCK]
    c = Cache(8, lens, KV, D, BLOCK)
    starts, counts = [0, 0, 37, BLOCK], [0, 1, 63, 2 * BLOCK]
    W = max(counts) + 3
    ko, vo = (torch.full((4, KV, W, D), 7.0, dtype=DT[fmt], device="cuda") for _ in range(2))
    st = ints([0])
    plan = pa.Q8ReadPlan(*c.cuda(), ints(starts), counts=ints(counts), k_out=ko, v_out=vo, status=st)
    plan.run()
    torch.cuda.synchronize()
    assert int(st) == 0
    for b in range(4):
        ids = np.arange(starts[b], starts[b] + counts[b])
        for h in range(KV):
            for got, cache, scale in ((ko, c.kc, c.ks), (vo, c.vc, c.vs)):
                p = c.table[b, ids // BLOCK]
                want = torch.from_numpy(cache[p, ids % BLOCK, h].astype(np.float32) * scale[p, h][:, None]).to(DT[fmt])
                assert torch.equal(got[b, h, : counts[b]].cpu(), want)
                assert bool((got[b, h, counts[b]:] == 7).all())


@pytest.mark.gpu
def test_read_out_of_range(pa):
    c = Cache(9, [40, 40], 2, 64, 16)
    c.table[1, 1] = -1
    st = ints([0])
    ko, _ = pa.cache_read_q8(*c.cuda(), ints([-3, 0]), width=80, dtype=torch.float32, status=st)
    torch.cuda.synchronize()
    assert int(st) == 3
    assert bool((ko[0, :, :48] != 0).any()) and bool((ko[0, :, 48:] == 0).all())
    assert bool((ko[1, :, 16:32] == 0).all()) and bool((ko[1, :, 32:48] != 0).any())


# ------------------------------------------------------------------ GPU: attention
def attend(pa, c, q, fmt, causal, scale=None, selected=None, counts=None, want_status=0):
    scale = float(np.float32(scale if scale is not None else c.D ** -0.5))
    st = ints([0])
    out = torch.full(q.shape, math.nan, dtype=DT[fmt], device="cuda")
    sel = {} if selected is None else dict(selected=ints(selected), counts=ints(counts))
    plan = pa.Q8Plan(q.cuda(), *c.cuda(), ints(c.lens), scale=scale, causal=causal, out=out, status=st, **sel)
    plan.run()
    first = out.clone()
    plan.run()
    torch.cuda.synchronize()
    assert int(st) == want_status
    assert torch.equal(out, first)  # and the workspace was left as it has to be
    want, tol = c.attend(as64(q), scale, causal, fmt, selected, counts)
    off = np.abs(as64(out) - want)
    assert np.all(off <= tol), f"{np.nanmax(off / np.maximum(tol, 1e-300))} of the bound"
    return out


SHAPES = [  # D, BLOCK, KV, G, NQ
    (64, 8, 1, 1, 1), (128, 8, 2, 4, 1), (64, 16, 2, 8, 1), (128, 16, 2, 4, 2), (64, 32, 3, 3, 3), (128, 32, 1, 8, 2), (64, 64, 2, 5, 4),
    (128, 64, 1, 2, 16), (64, 16, 1, 7, 7), (128, 16, 1, 33, 1), (64, 8, 1, 16, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_attention(pa, fmt, shape):
    D, BLOCK, KV, G, NQ = shape
    lens = [0, 1, 2, NQ, BLOCK - 1, BLOCK, BLOCK + 1, 127, 128, 129, 700]
    c = Cache(10, lens, KV, D, BLOCK)
    q = rows_of(c.rng, fmt, len(lens), KV * G, NQ, D) * 2
    for causal in (False, True):
        attend(pa, c, q, fmt, causal)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
def test_attention_over_many_pieces(pa, fmt):
    for lens, KV, G, NQ, D, BLOCK in (([16001], 1, 4, 1, 128, 16), ([9000, 3], 2, 8, 4, 64, 32), ([5000] * 3 + [40] * 30, 2, 4, 1, 64, 8)):
        c = Cache(11, lens, KV, D, BLOCK)
        attend(pa, c, rows_of(c.rng, fmt, len(lens), KV * G, NQ, D) * 2, fmt, True)


@pytest.mark.gpu
@pytest.mark.parametrize("B,KV", [(3, 8), (6, 8), (10, 8), (14, 8), (19, 8), (38, 8), (60, 8), (9, 7), (40, 1), (150, 1), (152, 2)])
def test_attention_of_uneven_batches(pa, B, KV):
    """Lengths from even to a single long one: whole sequences, equal pieces and shared ranges."""
    rng = np.random.default_rng(B)
    for uneven in (0, 1, 4, 20):
        lens = np.ceil(rng.random(B) ** uneven * (60000 / (B * KV) + 200)).astype(int)
        lens[rng.integers(B)] = 0
        c = Cache(30 + uneven, lens.tolist(), KV, 64, 16)
        attend(pa, c, rows_of(c.rng, "f16", B, KV, 1, 64) * 2, "f16", False)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,KV,D,BLOCK,G,NQ", [(330, 1, 64, 8, 3, 2), (60, 8, 128, 16, 1, 1), (700, 1, 128, 32, 2, 1), (41, 8, 64, 64, 2, 4)])
def test_attention_of_many_short_sequences(pa, fmt, B, KV, D, BLOCK, G, NQ):
    """More sequences and heads than CTAs, each short, some empty, some longer than the rest; all blocks, and lists of some."""
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 130, B)
    lens[rng.integers(0, B, 9)] = 0
    for longest in (130, 700):
        lens[rng.integers(0, B, 3)] = longest
        c = Cache(31, lens.tolist(), KV, D, BLOCK)
        q = rows_of(c.rng, fmt, B, KV * G, NQ, D) * 2
        attend(pa, c, q, fmt, True)
    sel, cnt = c.select(q.float().numpy(), 2, 0, 1)
    attend(pa, c, q, fmt, False, selected=sel, counts=cnt)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
def test_attention_with_scales_of_every_size(pa, fmt):
    """Value scales over many powers of two, zeros among them; the weight on small and large ones alike."""
    lens = [300, 77]
    c = Cache(12, lens, 2, 128, 16)
    c.vs = np.exp2(c.rng.integers(-30, 10, c.vs.shape)).astype(np.float32)
    c.vs[c.table[0, 3]] = 0
    c.vs[c.table[1, 1]] = 2.0 ** -120
    c.ks[c.table[0, 5]] = 0
    if fmt == "f16":
        c.vs = np.minimum(c.vs, 2.0 ** 6)
    q = rows_of(c.rng, fmt, 2, 8, 1, 128) * 6  # peaked: single keys take most of the weight
    attend(pa, c, q, fmt, False)
    c.vs[:] = np.float32(2.0 ** -90)
    if fmt != "f16":
        attend(pa, c, q, fmt, False)


@pytest.mark.gpu
def test_attention_of_queries_of_every_size(pa):
    c = Cache(13, [200] * 4, 1, 64, 16)
    q = rows_of(c.rng, "f32", 4, 8, 1, 64)
    for i, e in enumerate((2.0 ** -140, 2.0 ** -60, 1.0, 0.0)):
        q[:, i] *= e
    q[:, 4, :, 0] = 1e30   # one channel over all others: its sign decides
    q[0, 5], q[1, 5] = 0, 3e-39
    attend(pa, c, q[:, :4].contiguous(), "f32", False, scale=0.2)
    attend(pa, c, q.clamp(-1e4, 1e4), "f32", False, scale=1e-3)
    for fmt in ("f16", "bf16"):
        attend(pa, c, q.clamp(-1e4, 1e4).to(DT[fmt]), fmt, False, scale=1e-3)
    # large scores: the softmax is one key
    for fmt in DT:
        x = rows_of(c.rng, fmt, 4, 8, 1, 64) * 300
        out = pa.decode_q8(x.cuda(), *c.cuda(), ints(c.lens), scale=1.0)
        torch.cuda.synchronize()
        for b in range(4):
            K, V = c.rows(b, np.arange(200), 0)
            s = np.sort(as64(x)[b, :, 0] @ K.T, 1)
            top = (as64(x)[b, :, 0] @ K.T).argmax(1)
            for h in range(8):
                if s[h, -1] - s[h, -2] > 40:
                    np.testing.assert_allclose(as64(out)[b, h, 0], V[top[h]], rtol=2.0 ** -7, atol=1e-6)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "bf16"])
@pytest.mark.parametrize("G", [4, 20])
def test_attention_of_queries_near_the_largest_number(pa, fmt, G):
    """Factors of rows and keys stay finite: the softmax is one key, and no output is a NaN."""
    c = Cache(27, [200] * 2, 1, 64, 16)
    x = rows_of(c.rng, fmt, 2, G, 1, 64)
    out = pa.decode_q8((x * 2.0 ** 120).cuda(), *c.cuda(), ints(c.lens), scale=0.125)
    torch.cuda.synchronize()
    for b in range(2):
        K, V = c.rows(b, np.arange(200), 0)
        np.testing.assert_allclose(as64(out)[b, :, 0], V[(as64(x)[b, :, 0] @ K.T).argmax(1)], rtol=2.0 ** -7, atol=1e-6)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
def test_attention_with_the_smallest_key_scales(pa, fmt):
    """A key scale below 2^-96 counts as 2^-96, also where the queries are large enough to tell."""
    c = Cache(28, [200] * 2, 1, 64, 16)
    c.ks[:] = np.float32(2.0 ** -96)
    c.ks[c.table[0, :5]] = 0
    c.ks[c.table[1, 3:]] = np.float32(2.0 ** -110)
    q = rows_of(c.rng, fmt, 2, 4, 1, 64)
    if fmt != "f16":
        q = q * 2.0 ** 90
        attend(pa, c, q, fmt, True)
    attend(pa, c, q, fmt, True, scale=2.0 ** 20)


@pytest.mark.gpu
def test_attention_of_what_is_not_finite(pa):
    """A query row that is not finite is its own concern."""
    c = Cache(14, [100], 1, 64, 16)
    for fmt in DT:
        q = rows_of(c.rng, fmt, 1, 8, 1, 64)
        clean = attend(pa, c, q, fmt, False)
        q[0, 3, 0, 7] = math.nan
        out = pa.decode_q8(q.cuda(), *c.cuda(), ints(c.lens), scale=0.125)
        torch.cuda.synchronize()
        assert bool(out[0, 3].isnan().all())
        keep = [i for i in range(8) if i != 3]
        assert torch.equal(out[:, keep], clean[:, keep])


@pytest.mark.gpu
def test_bad_blocks_and_lengths(pa):
    """Entries outside the pool are left out and reported; scales of blocks that nobody sees may be anything."""
    c = Cache(15, [100, 90], 2, 64, 16, width=8)
    q = rows_of(c.rng, "f16", 2, 8, 1, 64)
    c.table[0, 2], c.table[1, 0] = -5, 10 ** 7
    c.table[:, 7] = 2 ** 30  # behind the lengths: not looked at
    unseen = [p for p in range(len(c.ks)) if p not in c.table]
    c.ks[unseen], c.vs[unseen] = math.nan, math.inf
    st = ints([0])
    out = pa.decode_q8(q.cuda(), *c.cuda(), ints(c.lens), scale=0.125, status=st)
    torch.cuda.synchronize()
    assert int(st) == 1
    good = [np.setdiff1d(np.arange(7), [2]), np.arange(1, 6)]
    sel, cnt = np.full((2, 2, 7), -1), np.zeros((2, 2))
    for b in range(2):
        sel[b, :, : len(good[b])], cnt[b] = good[b], len(good[b])
    want, tol = c.attend(as64(q), 0.125, False, "f16", sel.astype(int), cnt.astype(int))
    assert np.all(np.abs(as64(out) - want) <= tol)
    c = Cache(15, [100, 90], 2, 64, 16, width=8)
    st.zero_()
    out = pa.decode_q8(q.cuda(), *c.cuda(), ints([-7, 5000]), scale=0.125, status=st)
    torch.cuda.synchronize()
    assert int(st) == 2 and bool((out[0] == 0).all())
    c.lens = np.array([0, 128], np.int32)
    want, tol = c.attend(as64(q), 0.125, False, "f16")
    assert np.all(np.abs(as64(out) - want) <= tol)


# ------------------------------------------------------------------ GPU: selection
def selection(pa, c, q, budget, first, last, want_status=0):
    st, db = ints([0]), torch.from_numpy(c.bounds).cuda()
    dev = c.cuda()
    plan = pa.Q8SelectPlan(q.cuda(), db, dev[2], dev[4], ints(c.lens), BLOCK=c.BLOCK, budget=budget, keep_first=first, keep_last=last,
                           status=st)
    plan.selected.fill_(-99)
    plan.run()
    torch.cuda.synchronize()
    want = c.select(q.float().numpy(), budget, first, last)
    np.testing.assert_array_equal(plan.selected.cpu().numpy(), want[0])
    np.testing.assert_array_equal(plan.counts.cpu().numpy(), want[1])
    assert int(st) == want_status
    return want


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_selection(pa, fmt, shape):
    D, BLOCK, KV, G, NQ = shape
    lens = [0, 1, BLOCK, 5 * BLOCK, 5 * BLOCK + 1, 6 * BLOCK, 40 * BLOCK - 3, 200]
    c = Cache(16, lens, KV, D, BLOCK)
    q = rows_of(c.rng, fmt, len(lens), KV * G, NQ, D)
    for budget, first, last in ((5, 1, 1), (5, 0, 0), (1, 0, 1), (1, 0, 0), (5, 2, 3), (17, 1, 4), (100, 0, 1)):
        sel, cnt = selection(pa, c, q, budget, first, last)
        if budget in (5, 17) and first == 1:
            attend(pa, c, q, fmt, True, selected=sel, counts=cnt)


@pytest.mark.gpu
def test_selection_of_long_sequences(pa):
    """Clusters of every size, more candidates than threads, few sequences and many."""
    for B, KV, n, BLOCK in ((1, 1, 40000, 8), (1, 8, 5000, 8), (5, 8, 3000, 8), (30, 3, 2200, 8), (200, 2, 1500, 16)):
        c = Cache(17, [n - 7 * b for b in range(B)], KV, 64, BLOCK)
        q = rows_of(c.rng, "f16", B, KV * 2, 1, 64)
        nb = -(-n // BLOCK)
        for budget in (nb // 7, nb - 3):
            selection(pa, c, q, budget, 2, 3)


@pytest.mark.gpu
@pytest.mark.parametrize("B,KV,D,G,NQ,maxb", [(60, 8, 128, 2, 1, 30), (310, 1, 64, 3, 2, 65), (40, 8, 128, 40, 4, 20), (306, 1, 128, 1, 1, 4096), (306, 1, 64, 2, 1, 4097)])
def test_selection_of_many_sequences(pa, B, KV, D, G, NQ, maxb):
    """More sequences and heads than two CTAs an SM; short and long ones, some empty."""
    rng = np.random.default_rng(B + D)
    lens = rng.integers(0, min(maxb, 60) * 8, B)
    lens[:3] = 0, 1, maxb * 8
    pool = 500
    c = Cache(32, [8], KV, D, 8)
    c.bounds = np.sort(rng.integers(-127, 128, (pool, KV, 2, D)).astype(np.int8), 2)
    c.ks = rng.random((pool, KV)).astype(np.float32)
    c.table, c.lens = rng.integers(0, pool, (B, maxb)).astype(np.int32), lens.astype(np.int32)
    q = rows_of(rng, "f16", B, KV * G, NQ, D)
    st = ints([0])
    sel, cnt = pa.select_blocks_q8(q.cuda(), torch.from_numpy(c.bounds).cuda(), torch.from_numpy(c.ks).cuda(), ints(c.table), ints(c.lens),
                                   BLOCK=8, budget=7, keep_first=1, keep_last=2, status=st)
    torch.cuda.synchronize()
    ws, wc = c.select(q.float().numpy(), 7, 1, 2)
    np.testing.assert_array_equal(sel.cpu().numpy(), ws)
    np.testing.assert_array_equal(cnt.cpu().numpy(), wc)
    assert int(st) == 0


@pytest.mark.gpu
def test_selection_of_equal_scores(pa):
    """Ties: the lowest blocks; all scores zero, all but a few equal, scales that are no numbers."""
    c = Cache(18, [1000, 990], 2, 64, 16)
    q = rows_of(c.rng, "f16", 2, 4, 1, 64)
    selection(pa, c, torch.zeros_like(q), 20, 1, 2)
    c.bounds[:] = c.bounds[:1, :1]
    c.ks[:] = np.float32(0.25)
    selection(pa, c, q, 20, 1, 2)
    for p in c.table[0, 30:33]:
        c.ks[p] = 0.5
    selection(pa, c, q, 20, 1, 2)
    selection(pa, c, q, 61, 0, 0)
    c.ks[c.table[0, 5:20]] = math.nan
    c.ks[c.table[1, 50:60]] = math.inf
    # a NaN is lower than any other
    want = np.full((2, 2, 30), -1)
    for h in range(2):
        want[0, h] = np.sort(np.concatenate(([30, 31, 32], [i for i in range(63) if not 5 <= i < 20 and i not in (30, 31, 32)][:27])))
        want[1, h] = np.concatenate((np.arange(20), np.arange(50, 60)))
    dev = c.cuda()
    sel, _ = pa.select_blocks_q8(q.cuda(), torch.from_numpy(c.bounds).cuda(), dev[2], dev[4], ints(c.lens), BLOCK=16, budget=30, keep_last=0)
    torch.cuda.synchronize()
    got = sel.cpu().numpy()
    for h in range(2):
        np.testing.assert_array_equal(got[0, h], want[0, h])
        np.testing.assert_array_equal(got[1, h], want[1, h])


@pytest.mark.gpu
def test_selection_with_bad_blocks(pa):
    c = Cache(19, [400], 1, 64, 16)
    c.table[0, 7] = 10 ** 6
    q = rows_of(c.rng, "f16", 1, 1, 1, 64)
    st, dev = ints([0]), c.cuda()
    sel, cnt = pa.select_blocks_q8(q.cuda(), torch.from_numpy(c.bounds).cuda(), dev[2], dev[4], ints(c.lens), BLOCK=16, budget=24,
                                   keep_first=0, keep_last=0, status=st)
    torch.cuda.synchronize()
    assert int(st) == 1 and sel[0, 0].tolist() == [i for i in range(25) if i != 7] and int(cnt) == 24


@pytest.mark.gpu
def test_selected_lists_of_a_callers_own(pa):
    """Lists in any order, with places left out, none at all, entries behind the sequence, the same block twice."""
    c = Cache(20, [130, 64, 50, 0], 2, 64, 16)
    q = rows_of(c.rng, "f32", 4, 4, 2, 64)
    sel = np.full((4, 2, 9), -1)
    sel[0, 0, :5] = [7, -1, 0, 8, 3]
    sel[0, 1, :9] = [8, 7, 6, 5, 4, 3, 2, 1, 0]
    sel[1, 0, :2] = [3, 1]
    sel[2, 0, :3] = [2, 2, 0]
    sel[3, 1, :1] = [0]
    cnt = np.array([[5, 9], [2, 0], [3, 4], [0, 1]])
    attend(pa, c, q, "f32", True, selected=sel, counts=cnt, want_status=1)  # block 0 of the empty sequence
    sel[3] = -1
    sel[1, 1, 0] = 77
    cnt[1, 1] = 1
    attend(pa, c, q, "f32", False, selected=sel, counts=cnt, want_status=1)
    sel[1, 1, 0] = -1
    attend(pa, c, q, "f32", False, selected=sel, counts=cnt)
    st = ints([0])
    pa.decode_q8(q.cuda(), *c.cuda(), ints(c.lens), scale=0.1, selected=ints(sel), counts=ints(cnt - 1), status=st)
    torch.cuda.synchronize()
    assert int(st) == 2  # a count below zero


# ------------------------------------------------------------------ GPU: refusals of the binding
@pytest.mark.gpu
def test_refused_tensors(pa):
    c = Cache(21, [20, 30], 2, 64, 16)
    dev, lens = c.cuda(), ints(c.lens)
    q, kn = torch.randn(2, 4, 1, 64, device="cuda").half(), torch.randn(2, 2, 1, 64, device="cuda").half()
    bounds = torch.from_numpy(c.bounds).cuda()
    calls = {
        "append": lambda **k: pa.cache_append_q8(**{**dict(k_new=kn, v_new=kn.clone(), k_cache=dev[0], v_cache=dev[1], k_scale=dev[2], v_scale=dev[3],
                                                           block_table=dev[4], seq_lens=lens), **k}),
        "read": lambda **k: pa.cache_read_q8(**{**dict(k_cache=dev[0], v_cache=dev[1], k_scale=dev[2], v_scale=dev[3], block_table=dev[4],
                                                       starts=lens, width=4), **k}),
        "select": lambda **k: pa.select_blocks_q8(**{**dict(q=q, bounds=bounds, k_scale=dev[2], block_table=dev[4], seq_lens=lens, BLOCK=16,
                                                            budget=2), **k}),
        "decode": lambda **k: pa.decode_q8(**{**dict(q=q, k_cache=dev[0], v_cache=dev[1], k_scale=dev[2], v_scale=dev[3], block_table=dev[4],
                                                     seq_lens=lens, scale=0.1), **k}),
    }
    for f in calls.values():
        f()
    for name, bad in [("append", dict(k_cache=dev[0].float())), ("append", dict(k_new=kn[:, :1])), ("append", dict(v_new=kn.float())),
                      ("append", dict(k_scale=dev[2].half())), ("append", dict(k_scale=dev[2][:1])), ("append", dict(counts=lens.long())),
                      ("append", dict(bounds=bounds[:, :, :1])), ("append", dict(seq_lens=lens.cpu())), ("append", dict(k_new=kn.cpu())),
                      ("append", dict(k_new=torch.randn(2, 2, 1, 128, device="cuda").half()[..., ::2])),
                      ("read", dict(dtype=torch.int8)), ("read", dict(starts=lens[:1])), ("read", dict(v_cache=dev[1][:, :, :1])),
                      ("select", dict(budget=0)), ("select", dict(q=q.long())), ("select", dict(block_table=dev[4][:1])),
                      ("select", dict(k_scale=dev[2].t().contiguous().t())),
                      ("select", dict(budget=2 ** 32)), ("decode", dict(q=q[..., :32])), ("decode", dict(selected=lens.view(2, 1, 1))),
                      ("decode", dict(out=torch.zeros(2, 4, 1, 64, device="cuda"))), ("decode", dict(out=torch.zeros(2, 4, 1, 64).half())),
                      ("decode", dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8))), ("decode", dict(q=q.double())),
                      ("decode", dict(status=torch.zeros(1, device="cuda")))]:
        with pytest.raises((ValueError, TypeError)):
            calls[name](**bad)
    with pytest.raises(pa.PagedAttentionError):
        calls["decode"](workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))
