"""Decode attention with modified scores and the weight each key got
(include/pa_scored.h): refusals on the CPU, the kernels against 64-bit
arithmetic on the GPU.

Error bound.  With delta_j an upper bound on the error of key j's score
(natural units), the softmax weight p_j is off by at most p_j (delta_j +
sum_k p_k delta_k) to first order, doubled here for the higher ones.
  delta_j = 2^-23 (D scale sum |q k| + 4 |t_j| + 4 |bias_j|): the float32 dot
  of D terms, tanh, products and the base-2 change, the bias of the distance.
The weights themselves (exp2, sums over keys): 2^-20 of them.  P is used as a
16-bit high part plus remainder: 2^-16 (bf16), 2^-21 (fp16, and 2^-25 of the
row's largest weight per key where the remainder leaves fp16's range).  Then
half a step of the output's type.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_182_gb300 import _build

    _build.build()
    from paged_kv_cache_182_gb300 import binding

    return binding


# ------------------------------------------------------------------ reference
def visible(i, j, total, causal, window, prefix):
    """The rule of include/pa_scored.h, for one row and an array of keys."""
    seen = np.abs(i - j) < window if window else np.ones(len(j), bool)
    if causal:
        seen &= j <= i
    return (seen | (j < prefix)) & (j < total)


def reference(x, kw):
    """(out, out bound, weights, weights bound) in 64 bits."""
    q, kc, vc, table, lens, kn, vn = (t.cpu() for t in x)
    f = lambda t: t.double().numpy()  # noqa: E731
    B, H, NQ, D = q.shape
    KV, bs = kc.shape[2], kc.shape[1]
    G, scale = H // KV, kw["scale"]
    cap, window, fmt = kw.get("softcap", 0.0), kw.get("window", 0), kw["fmt"]
    slopes = None if kw.get("slopes") is None else f(kw["slopes"].cpu())
    prefix = [0] * B if kw.get("prefix") is None else kw["prefix"].tolist()
    out, bound = np.zeros((B, H, NQ, D)), np.zeros((B, H, NQ, D))
    width = table.shape[1] * bs
    w, wb = np.zeros((B, width)), np.zeros((B, width))
    flat = [f(t.reshape(-1, KV, D)) for t in (kc, vc)]
    q, kn, vn = f(q), f(kn), f(vn)
    for b in range(B):
        n = min(max(int(lens[b]), 0), width)
        j = np.arange(n)
        slots = table[b].numpy()[j // bs].astype(np.int64) * bs + j % bs
        keys, m = np.arange(n + NQ), min(n + NQ, width)
        for h in range(H):
            K = np.concatenate((flat[0][slots, h // G], kn[b, h // G]))
            V = np.concatenate((flat[1][slots, h // G], vn[b, h // G]))
            for r in range(NQ):
                i = n + r
                t = scale * (K @ q[b, h, r])
                mag = D * scale * (np.abs(K) @ np.abs(q[b, h, r]))
                if cap:
                    t = cap * np.tanh(t / cap)
                bias = np.zeros(n + NQ) if slopes is None else slopes[h] * np.abs(i - keys)
                seen = visible(i, keys, n + NQ, kw.get("causal", False), window, prefix[b])
                assert seen.any()
                s = np.where(seen, t - bias, -np.inf)
                p = np.exp(s - s.max())
                p /= p.sum()
                delta = 2.0 ** -23 * (mag + 4 * np.abs(t) + 4 * np.abs(bias))
                both = p * (delta + (p * delta).sum()) * 2 + p * 2.0 ** -20
                Vs = np.where(seen[:, None], V, 0.0)
                out[b, h, r] = p @ Vs
                split = {"f32": 0.0, "f16": 2.0 ** -21, "bf16": 2.0 ** -16}[fmt]
                small = 2.0 ** -25 * p.max() if fmt == "f16" else 0.0
                e = (both + p * split + small * seen) @ np.abs(Vs)
                bound[b, h, r] = e + 2.0 ** -22 * (p @ np.abs(Vs))
                w[b, :m] += p[:m]
                wb[b, :m] += both[:m] + 2.0 ** -22 * p[:m]
    return out, bound, w, wb


def make(seed, fmt, lens, H, KV, D, BLOCK, NQ, poison=True, extra=0):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    maxb = max(1, max(-(-n // BLOCK) for n in lens)) + extra
    pool = sum(-(-n // BLOCK) for n in lens) + 2
    perm = torch.randperm(pool, generator=g).to(torch.int32)
    table = torch.full((B, maxb), -1, dtype=torch.int32)
    r = lambda *s: torch.randn(*s, generator=g).to(DT[fmt])  # noqa: E731
    kc, vc = r(pool, BLOCK, KV, D), r(pool, BLOCK, KV, D)
    at = 0
    used = torch.zeros(pool, BLOCK, dtype=torch.bool)
    for b, n in enumerate(lens):
        nb = -(-n // BLOCK)
        table[b, :nb] = perm[at:at + nb]
        at += nb
        for k in range(nb):
            used[table[b, k].long(), : min(BLOCK, n - k * BLOCK)] = True
    if poison:
        kc[~used] = math.nan
        vc[~used] = math.nan
    x = [2 * r(B, H, NQ, D), kc, vc, table, torch.tensor(lens, dtype=torch.int32), r(B, KV, NQ, D), r(B, KV, NQ, D)]
    return [t.cuda() for t in x], g


def compare(pa, x, kw, weights=True, **more):
    fmt = kw["fmt"]
    call = {k: v for k, v in kw.items() if k != "fmt"}
    width = x[3].shape[1] * x[1].shape[1]
    win = torch.rand(x[0].shape[0], width, generator=torch.Generator().manual_seed(1)).cuda()
    out, bound, w, wb = reference(x, kw)
    got = pa.decode_scored(*x, **call, **more)
    assert torch.isfinite(got.float()).all()
    o = got.double().cpu().numpy()
    lim = bound + HALF_STEP[{torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}[got.dtype]] * (np.abs(out) + bound)
    if got.dtype == torch.float16:
        lim += 2.0 ** -25
    assert np.all(np.abs(o - out) <= lim), float(np.max(np.abs(o - out) / lim))
    if not weights:
        return got
    wout = torch.full((x[0].shape[0], width), 7.0, device="cuda")
    got2, kw_out = pa.decode_scored(*x, **call, key_weights=win, key_weights_out=wout, decay=0.75, **more)
    torch.cuda.synchronize()
    assert kw_out is wout and torch.equal(got2, got)
    a = wout.double().cpu().numpy()
    old = 0.75 * win.double().cpu().numpy()
    for b, n in enumerate(x[4].tolist()):
        n = min(max(n, 0), width)
        m = min(n + x[0].shape[2], width)
        want, lim = w[b, :m].copy(), wb[b, :m] + 2.0 ** -149
        want[:n] += old[b, :n]
        lim[:n] += 2.0 ** -23 * old[b, :n]
        lim += 2.0 ** -23 * np.abs(want)
        assert np.all(np.abs(a[b, :m] - want) <= lim), (b, float(np.max(np.abs(a[b, :m] - want) / lim)))
        assert np.all(a[b, m:] == 7.0)  # behind the last key: left as it was
    return got


# ------------------------------------------------------------------ CPU: refusals
A = 1 << 24


def call(pa, score=True, weights=None, B=2, H=4, KV=2, D=64, BLOCK=16, NQ=1, scale=0.125, softcap=0.0, window=0, slopes=None,
         prefix=None, **o):
    opts = dict(batch=B, max_blocks=8, num_blocks=64, dtype=1, out_dtype=-1, partitions=0, workspace=20 * A, workspace_bytes=1 << 30)
    opts.update(o)
    s = pa.Score(softcap=softcap, window=window, slopes=slopes, prefix=prefix)
    w = None if weights is None else pa.KeyWeights(**{**dict(in_=30 * A, out=31 * A, decay=0.5, scratch=32 * A, scratch_bytes=1 << 30), **weights})
    p = [ctypes.c_void_p((i + 1) * A) for i in range(8)]
    return pa.LIB.pa_decode_scored(*p, ctypes.c_float(scale), H, KV, D, BLOCK, NQ, 1, ctypes.byref(s) if score else None,
                                   None if w is None else ctypes.byref(w), ctypes.byref(pa.PaOpts(**opts)), None)


NULL, DIMS, UNSUP, ALIGN, WS = -1, -2, -3, -4, -5


@pytest.mark.parametrize("kw,code", [
    (dict(score=False), NULL), (dict(softcap=-1.0), DIMS), (dict(softcap=math.inf), DIMS), (dict(softcap=math.nan), DIMS),
    (dict(window=-1), DIMS), (dict(weights=dict(decay=math.nan)), DIMS), (dict(partitions=2), UNSUP), (dict(merge_kernel=1), UNSUP),
    (dict(softcap=1e-40), DIMS), (dict(weights=dict(in_=31 * A + 64)), DIMS), (dict(slopes=A + 2), ALIGN), (dict(prefix=A + 1), ALIGN), (dict(weights=dict(out=None)), NULL),
    (dict(weights=dict(scratch=None)), WS), (dict(weights=dict(scratch_bytes=100)), WS), (dict(weights=dict(scratch=32 * A + 64)), ALIGN),
    (dict(weights=dict(out=31 * A + 2)), ALIGN), (dict(weights={}, NQ=17), UNSUP), (dict(NQ=17), UNSUP), (dict(H=5), DIMS),
    (dict(weights={}, H=5), DIMS), (dict(D=96), UNSUP), (dict(scale=math.nan), DIMS), (dict(workspace_bytes=10), WS),
    (dict(weights={}, B=5000), UNSUP), (dict(B=-1), DIMS),
])
def test_refusals(pa, kw, code):
    assert call(pa, **kw) == code


def test_empty_batch_and_scratch_sizes(pa):
    assert call(pa, B=0) == 0 and call(pa, B=0, weights={}) == 0
    f = pa.LIB.pa_scored_scratch_bytes
    assert f(2, 8, 16, 4, 2, 3) == 256 + 2 * 4 * 3 * (8 * 16 + 3) * 4
    assert f(0, 8, 16, 4, 2, 1) == f(2, 8, 16, 4, 3, 1) == f(2, 8, 16, 4, 2, 17) == f(4096, 1 << 25, 16, 1 << 30, 2, 16) == 0


# ------------------------------------------------------------------ GPU
SHAPES = [  # lens, H, KV, D, BLOCK, NQ
    ([0], 1, 1, 64, 16, 1), ([1, 2, 15, 16, 17], 4, 2, 64, 16, 1), ([700, 3, 129], 8, 2, 128, 16, 1), ([300, 257], 12, 4, 64, 32, 2),
    ([520, 64, 1], 6, 2, 128, 64, 4), ([400, 33], 10, 2, 128, 8, 4), ([900, 130], 16, 2, 64, 32, 16), ([260], 5, 1, 128, 32, 7),
    ([1500, 1024, 2], 3, 3, 128, 16, 1),
]
MODS = [
    dict(softcap=5.0), dict(slopes=True), dict(window=1), dict(window=100), dict(window=300, prefix=70), dict(prefix=2 ** 31 - 1),
    dict(softcap=20.0, slopes=True, window=130, prefix=20), dict(window=2 ** 31 - 1, prefix=-3),
]


def modified(mod, B, H, scale, fmt, causal):
    kw = dict(scale=scale, causal=causal, fmt=fmt, softcap=mod.get("softcap", 0.0), window=mod.get("window", 0))
    if mod.get("slopes"):
        kw["slopes"] = (2.0 ** (-6.0 * (torch.arange(H) + 1.0) / H)).float().cuda()
    if "prefix" in mod:
        kw["prefix"] = (torch.tensor([mod["prefix"]] * B, dtype=torch.int64) - torch.arange(B)).to(torch.int32).cuda()
    return kw


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_matches_64_bits(pa, shape, fmt):
    lens, H, KV, D, BLOCK, NQ = SHAPES[shape]
    x, _ = make(shape, fmt, lens, H, KV, D, BLOCK, NQ, extra=shape % 2)
    for i, mod in enumerate(MODS):
        causal = (i + shape) % 3 != 0
        kw = modified(mod, len(lens), H, 1 / math.sqrt(D), fmt, causal)
        compare(pa, x, kw, partitions=int(i == 4), out_dtype=torch.float32 if i % 2 else None)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,H,KV,NQ", [(128, 4, 1, 1), (64, 8, 2, 1), (128, 16, 1, 3)])
def test_long_sequences_windows_and_splits(pa, D, H, KV, NQ, fmt):
    # several partitions a segment; windows whose gap covers many stages
    x, _ = make(5, fmt, [6000, 2500, 40], H, KV, D, 16, NQ)
    for mod in (dict(softcap=30.0, slopes=True), dict(window=700, prefix=300), dict(window=64, prefix=1), dict(window=5000)):
        compare(pa, x, modified(mod, 3, H, 1 / math.sqrt(D), fmt, True))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("H,KV,NQ", [(8, 1, 4), (16, 2, 7), (17, 1, 1), (6, 2, 16), (5, 1, 16)])
def test_many_rows(pa, H, KV, NQ, fmt):
    # 17 to 80 rows a KV head: two row groups a pass, up to three passes
    x, _ = make(H + NQ, fmt, [1000, 385, 2], H, KV, 128, 16, NQ)
    for i, mod in enumerate(MODS):
        compare(pa, x, modified(mod, 3, H, 128 ** -0.5, fmt, i % 2 == 0))


@pytest.mark.gpu
@pytest.mark.parametrize("D,H,KV,NQ", [(64, 12, 3, 16), (128, 10, 2, 7), (64, 5, 1, 13), (128, 3, 1, 11), (64, 9, 1, 16)])
def test_many_rows_of_float32(pa, D, H, KV, NQ):
    # 64, 35, 65, 33 and 144 rows a KV head: passes of 32
    x, _ = make(H + NQ, "f32", [300, 0, 97, 1200], H, KV, D, 16, NQ)
    for mod in (dict(softcap=20.0), dict(slopes=True, window=150, prefix=40), dict(softcap=5.0, slopes=True)):
        compare(pa, x, modified(mod, 4, H, 1 / math.sqrt(D), "f32", True))


@pytest.mark.gpu
def test_infinities_and_nans_in_hidden_keys_of_many_rows(pa):
    x, _ = make(14, "bf16", [700, 300], 16, 2, 128, 16, 4)
    kw = modified(dict(window=150, prefix=33), 2, 16, 0.09, "bf16", True)
    call = {k: v for k, v in kw.items() if k != "fmt"}
    want = pa.decode_scored(*x, **call)
    for b, n in enumerate([700, 300]):
        for j in range(33 - b, n - 149):
            phys = int(x[3][b, j // 16])
            x[1][phys, j % 16] = math.nan if j % 2 else math.inf
            x[2][phys, j % 16] = math.inf if j % 3 else math.nan
    assert torch.equal(pa.decode_scored(*x, **call), want)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,B,D,NQ", [("f16", 1500, 64, 1), ("bf16", 1500, 128, 16), ("f32", 1500, 64, 16), ("f16", 4096, 128, 1)])
def test_large_batches(pa, fmt, B, D, NQ):
    g = torch.Generator().manual_seed(B + D)
    lens = torch.randint(0, 60, (B,), generator=g).tolist()
    x, _ = make(B, fmt, lens, 2, 1, D, 16, NQ)
    kw = modified(dict(softcap=9.0, window=21, prefix=2 ** 20), B, 2, 0.1, fmt, True)
    kw["prefix"] = (torch.arange(B) % 9).to(torch.int32).cuda()
    some = list(range(0, B, 97))  # the reference for some sequences
    out, w = pa.decode_scored(*x, **{k: v for k, v in kw.items() if k != "fmt"},
                              key_weights_out=torch.zeros(B, x[3].shape[1] * 16, device="cuda"))
    torch.cuda.synchronize()
    part = [x[0][some], x[1], x[2], x[3][some], x[4][some], x[5][some], x[6][some]]
    want, bound, ww, wb = reference(part, {**kw, "prefix": kw["prefix"][some]})
    o = out[some].double().cpu().numpy()
    assert np.all(np.abs(o - want) <= bound + HALF_STEP[fmt] * (np.abs(want) + bound) + 2.0 ** -25)
    assert np.all(np.abs(w[some].double().cpu().numpy() - ww) <= wb + 2.0 ** -23 * ww)


@pytest.mark.gpu
def test_scores_past_32_bits_of_offset(pa):
    # 2 x 8 heads x 16 rows of up to 16M tokens of capacity: 17 GB of scores
    x, _ = make(17, "f16", [70, 33], 8, 1, 64, 16, 16)
    wide = torch.full((2, 1 << 20), -1, dtype=torch.int32, device="cuda")
    wide[:, : x[3].shape[1]] = x[3]
    kw = dict(scale=0.1, causal=True, softcap=7.0)
    a, wa = pa.decode_scored(*x, **kw, key_weights_out=torch.zeros(2, x[3].shape[1] * 16, device="cuda"))
    x[3] = wide
    b, wb = pa.decode_scored(*x, **kw, key_weights_out=torch.zeros(2, 16 << 20, device="cuda"))
    assert torch.equal(a, b) and torch.equal(wa, wb[:, : wa.shape[1]]) and float(wb[:, 100:].abs().max()) == 0.0


@pytest.mark.gpu
def test_without_modification_equals_decode(pa):
    x, _ = make(2, "f16", [300, 77, 1300], 8, 2, 128, 16, 2)
    plain = pa.decode(*x, scale=0.1, causal=True)
    got = pa.decode_scored(*x, scale=0.1, causal=True)
    assert torch.equal(plain, got)
    x, _ = make(2, "f16", [300, 77, 1300], 12, 1, 128, 16, 3)
    assert torch.equal(pa.decode(*x, scale=0.1, causal=True, kernel=1), pa.decode_scored(*x, scale=0.1, causal=True))


@pytest.mark.gpu
def test_infinities_and_nans_in_hidden_keys(pa):
    # rows that a window hides hold NaN and infinities; neither the output nor a weight may see them
    for fmt in ("f16", "f32"):
        x, _ = make(4, fmt, [500, 260], 4, 2, 64, 16, 2)
        kw = modified(dict(window=100, prefix=33), 2, 4, 0.125, fmt, True)
        want = pa.decode_scored(*x, **{k: v for k, v in kw.items() if k != "fmt"})
        for b, n in enumerate([500, 260]):
            for j in range(33 - b, n - 99):
                phys = int(x[3][b, j // 16])
                x[1][phys, j % 16] = math.nan if j % 2 else math.inf
                x[2][phys, j % 16] = math.inf if j % 3 else math.nan
        got, w = pa.decode_scored(*x, **{k: v for k, v in kw.items() if k != "fmt"},
                                  key_weights_out=torch.zeros(2, x[3].shape[1] * 16, device="cuda"))
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        assert torch.isfinite(w).all() and float(w[0, 33:400].abs().max()) == 0.0
        # every head's and row's weights sum to one
        assert abs(float(w[0].double().sum()) - 8) < 8e-5


@pytest.mark.gpu
def test_weights_in_place_without_earlier_ones_and_repeated(pa):
    x, _ = make(6, "bf16", [200, 130], 8, 4, 128, 32, 1)
    kw = dict(scale=0.09, causal=True, softcap=10.0)
    zero = torch.zeros(2, x[3].shape[1] * 32, device="cuda")
    _, fresh = pa.decode_scored(*x, **kw, key_weights_out=zero.clone())
    acc = torch.rand(2, zero.shape[1], device="cuda")
    want = acc.clone()
    plan = pa.ScoredPlan(*x, **kw, key_weights=acc, decay=0.5)
    for _ in range(3):
        plan.run()
        for b, n in enumerate([200, 130]):
            want[b, :n] = torch.addcmul(fresh[b, :n], want[b, :n], torch.tensor(0.5, device="cuda"))
            want[b, n:n + 1] = fresh[b, n:n + 1]
    torch.cuda.synchronize()
    assert torch.allclose(acc, want, rtol=2.0 ** -21, atol=0.0)
    first = acc.clone()
    for _ in range(2):  # the same sums every time
        again = torch.zeros_like(zero)
        pa.decode_scored(*x, **kw, key_weights_out=again)
        assert torch.equal(again, fresh)
    assert torch.equal(first, acc)


@pytest.mark.gpu
def test_graph_replay_with_other_lengths_and_another_stream(pa):
    x, _ = make(8, "f16", [900, 400], 8, 2, 64, 32, 1, poison=False)
    kw = modified(dict(softcap=15.0, window=200, prefix=40), 2, 8, 0.125, "f16", True)
    call = {k: v for k, v in kw.items() if k != "fmt"}
    w = torch.zeros(2, x[3].shape[1] * 32, device="cuda")
    plan = pa.ScoredPlan(*x, **call, key_weights_out=w)
    plan.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
    for lens in ([900, 400], [17, 399], [500, 0]):
        x[4].copy_(torch.tensor(lens, dtype=torch.int32))
        w.zero_()
        graph.replay()
        torch.cuda.synchronize()
        out, weights = plan.out.clone(), w.clone()
        ref = torch.zeros_like(w)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got, _ = pa.decode_scored(*x, **call, key_weights_out=ref)
        side.synchronize()
        assert torch.equal(got, out) and torch.equal(ref, weights)
        compare(pa, x, kw)


@pytest.mark.gpu
def test_bad_lengths_and_blocks(pa):
    x, _ = make(9, "f16", [64, 64], 4, 2, 64, 16, 1, poison=False)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x[4].copy_(torch.tensor([-4, 1000], dtype=torch.int32))
    kw = modified(dict(window=20, prefix=3), 2, 4, 0.125, "f16", True)
    compare(pa, x, kw, weights=True, status=status)
    assert int(status) == pa.PA_STATUS_BAD_LENGTH
    x[4].fill_(64)
    x[3][0, 0] = x[1].shape[0]
    status.zero_()
    pa.decode_scored(*x, scale=0.125, window=64, status=status, checked=True)
    torch.cuda.synchronize()
    assert int(status) == pa.PA_STATUS_BAD_BLOCK


@pytest.mark.gpu
def test_refused_arguments(pa):
    x, _ = make(9, "f16", [64, 64], 4, 2, 64, 16, 1)
    for bad in (dict(slopes=torch.zeros(3, device="cuda")), dict(slopes=torch.zeros(4)), dict(prefix=torch.zeros(2, device="cuda")),
                dict(key_weights=torch.zeros(2, 63, device="cuda")), dict(key_weights_out=torch.zeros(2, 64, device="cuda").half())):
        with pytest.raises(ValueError):
            pa.decode_scored(*x, scale=0.1, **bad)
    with pytest.raises(pa.PagedAttentionError):
        pa.decode_scored(*x, scale=0.1, softcap=-2.0)


# ------------------------------------------------------------------ caps at the ends of float32's range
# scale / softcap subnormal, softcap * log2(e) infinite, scale / softcap near the ends, each with a scale that leaves the other fine
@pytest.mark.parametrize("softcap,scale", [(3e38, 0.125), (2.4e38, 1e10), (1e37, 0.125), (2e31, 0.125), (-3e38, 0.125), (1e-32, 0.125),
                                           (3e-38, -0.125), (1e-45, 0.125), (1.0, 1e-31)])
def test_refused_caps(pa, softcap, scale):
    assert call(pa, softcap=softcap, scale=scale) == DIMS and call(pa, softcap=softcap, scale=scale, weights={}) == DIMS
    assert call(pa, B=0, softcap=softcap, scale=scale) == DIMS


@pytest.mark.parametrize("softcap,scale", [(1e29, 0.125), (2.3e38, 1e10), (1e-30, 0.125), (50.0, 0.0), (50.0, -0.125), (0.0, 1e-31)])
def test_accepted_caps(pa, softcap, scale):
    assert call(pa, B=0, softcap=softcap, scale=scale) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f16", "f32"])
@pytest.mark.parametrize("cap", [1e6, 1e20, 1e29])
def test_caps_that_change_nothing(pa, fmt, cap):
    x, _ = make(32, fmt, [300, 41], 8, 2, 64, 16, 2)
    for mod in (dict(softcap=cap), dict(softcap=cap, slopes=True, window=90)):
        compare(pa, x, modified(mod, 2, 8, 0.125, fmt, True))


@pytest.mark.gpu
def test_a_decode_that_reads_its_inputs_early_behind_key_weights(pa):
    # the kernel ahead of the second call (the key weights') writes none of its inputs; the one before
    # that writes its q
    x, _ = make(41, "f16", [6000, 5000, 300], 16, 2, 128, 16, 1)
    zero = torch.zeros(3, x[3].shape[1] * 16, device="cuda")
    first = pa.ScoredPlan(*x, scale=0.09, causal=True, softcap=20.0, key_weights_out=zero)
    second = pa.Plan(first.out, *x[1:], scale=1.0, causal=True, inputs_unchanged=True)
    sets = [torch.randn_like(x[0]) for _ in range(2)]
    want = []
    for q in sets:
        x[0].copy_(q)
        first.run()
        torch.cuda.synchronize()
        want.append(second.run().clone())
        torch.cuda.synchronize()
    assert not torch.equal(*want)
    got = []
    for n in range(40):
        x[0].copy_(sets[n % 2])
        first.run()
        got.append(second.run().clone())
    torch.cuda.synchronize()
    for n, t in enumerate(got):
        assert torch.equal(t, want[n % 2]), n


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
def test_weights_of_two_schedules(pa, fmt):
    # split or whole, the weights agree up to the rounding of the softmax denominators
    x, _ = make(33, fmt, [9000, 700, 31], 4, 1, 128, 16, 1)
    for mod in (dict(softcap=20.0), dict(slopes=True, window=3000, prefix=50)):
        kw = modified(mod, 3, 4, 0.09, fmt, True)
        _, bound, want, lim = reference(x, kw)
        kw.pop("fmt")
        got = [pa.decode_scored(*x, **kw, partitions=n, key_weights_out=torch.zeros(3, x[3].shape[1] * 16, device="cuda"))[1]
               for n in (0, 1)]
        a, b = (t.double().cpu().numpy() for t in got)
        assert np.all(np.abs(a - b) <= 2 * (lim + 2.0 ** -23 * want))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,H,KV,D", [("f16", 4, 2, 64), ("f32", 4, 2, 64), ("bf16", 16, 2, 128), ("f16", 32, 2, 128), ("f32", 12, 1, 128)])
def test_hidden_keys_under_a_cap_change_nothing(pa, fmt, H, KV, D):
    # the way a block's tanh is computed goes by its largest score, hidden ones included: what hidden
    # keys hold (large, infinite, NaN) must not move a visible score by a bit
    lens = [500, 260, 113]
    x, _ = make(31, fmt, lens, H, KV, D, 16, 2)
    x[0] *= 0.02  # visible scores of every size below the cap
    kw = modified(dict(softcap=1.5, window=100, prefix=33), 3, H, 1 / math.sqrt(D), fmt, True)
    kw.pop("fmt")
    width = x[3].shape[1] * 16
    want, w = pa.decode_scored(*x, **kw, key_weights_out=torch.zeros(3, width, device="cuda"))
    for large in (1.0, 300.0, math.inf):
        for b, n in enumerate(lens):
            for j in range(33 - b, n - 99):
                phys = int(x[3][b, j // 16])
                x[1][phys, j % 16] = math.nan if large == math.inf and j % 2 else large
                x[2][phys, j % 16] = large if j % 3 else -large
        got, u = pa.decode_scored(*x, **kw, key_weights_out=torch.zeros(3, width, device="cuda"))
        assert torch.equal(got, want) and torch.equal(u, w)
