"""Gradient of attention with modified scores (pa_attention_vjp_scored):
refusals on the CPU; on the GPU against the formula in 64 bits and against
differences of the forward pass.

Error bounds, per element, with u the half step of the type that p and ds
take into the products (tensor cores: 2^-8 bf16, 2^-11 fp16; else 0):
  score error delta = 2^-23 (D scale sum |q k| + 4 |t| + 4 |bias|)
  p relative error  r = 2 (delta + sum_j p delta) + 2^-19
  ds error          E = |ds| (r + 2^-20) + p scale 2^-23 D (|g|.|v| + |y|.|g|) + p scale |dp - delta| 2^-20
  dv: (p (u + r))^T |g|;  dk: (|ds| u + E)^T |q|;  dq: (|ds| u + E) |k|
plus 2^-23 a term of each float32 sum, 2^-25 per p or ds below fp16's range,
and half a step of the output.
"""
import ctypes
import math

import numpy as np
import pytest
import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_182_gb300 import _build

    _build.build()
    from paged_kv_cache_182_gb300 import binding

    return binding


# ------------------------------------------------------------------ reference
def probabilities(q, k, b, h, kw, mask=None):
    """p, raw capped argument's tanh, score error bound; float64 of one head."""
    SQ, SK = len(q), len(k)
    i, j = np.arange(SQ)[:, None], np.arange(SK)[None, :]
    t = kw["scale"] * (q @ k.T)
    mag = q.shape[1] * abs(kw["scale"]) * (np.abs(q) @ np.abs(k).T)
    th = np.zeros_like(t)
    if kw.get("softcap"):
        th = np.tanh(t / kw["softcap"])
        t = kw["softcap"] * th
    bias = np.zeros_like(t)
    if kw.get("slopes") is not None:
        bias = float(kw["slopes"][h]) * np.abs(i - j)
    seen = np.ones((SQ, SK), bool)
    if kw.get("causal"):
        seen &= j <= i
    if kw.get("window"):
        seen &= np.abs(i - j) < kw["window"]
    if kw.get("prefix") is not None:
        seen |= j < int(kw["prefix"][b])
    s = np.where(seen, t - bias, -np.inf)
    if mask is not None:
        s = s + mask
    top = s.max(1, keepdims=True, initial=-np.inf)
    e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    tot = e.sum(1, keepdims=True)
    return e / np.where(tot == 0, 1.0, tot), th, 2.0 ** -23 * (mag + 4 * np.abs(t) + 4 * np.abs(bias))


def forward(q, k, v, kw, mask=None):
    G = q.shape[1] // k.shape[1]
    y = np.zeros_like(q)
    for b in range(q.shape[0]):
        for h in range(q.shape[1]):
            m = None if mask is None else np.broadcast_to(mask, (q.shape[0], q.shape[1], q.shape[2], k.shape[2]))[b, h]
            y[b, h] = probabilities(q[b, h], k[b, h // G], b, h, kw, m)[0] @ v[b, h // G]
    return y


def gradient(q, k, v, y, g, kw, u=0.0, tiny=0.0, mask=None):
    B, HQ, SQ, D = q.shape
    HK, SK = k.shape[1], k.shape[2]
    G = HQ // HK
    out = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)]
    err = [np.zeros(q.shape), np.zeros(k.shape), np.zeros(k.shape)]
    for b in range(B):
        for h in range(HQ):
            kh = h // G
            m = None if mask is None else np.broadcast_to(mask, (B, HQ, SQ, SK))[b, h]
            p, th, delta = probabilities(q[b, h], k[b, kh], b, h, kw, m)
            dp = g[b, h] @ v[b, kh].T
            dl = (y[b, h] * g[b, h]).sum(1, keepdims=True)
            part = p * (dp - dl) * kw["scale"]
            ds = part * (1 - th ** 2)
            r = 2 * (delta + (p * delta).sum(1, keepdims=True)) + 2.0 ** -19
            terms = np.abs(g[b, h]) @ np.abs(v[b, kh]).T + (np.abs(y[b, h]) * np.abs(g[b, h])).sum(1, keepdims=True)
            E = np.abs(ds) * (r + 2.0 ** -20) + p * kw["scale"] * 2.0 ** -23 * D * terms + np.abs(part) * 2.0 ** -20
            E = E + np.abs(ds) * u + tiny * (p > 0)
            P = p * (u + r) + tiny * (p > 0)
            n = 2.0 ** -23
            out[0][b, h] = ds @ k[b, kh]
            err[0][b, h] = (E + n * SK * np.abs(ds)) @ np.abs(k[b, kh])
            out[1][b, kh] += ds.T @ q[b, h]
            err[1][b, kh] += (E + n * SQ * G * np.abs(ds)).T @ np.abs(q[b, h])
            out[2][b, kh] += p.T @ g[b, h]
            err[2][b, kh] += (P + n * SQ * G * p).T @ np.abs(g[b, h])
    return out, err


def make(seed, fmt, B, HQ, HK, SQ, SK, D):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(DT[fmt])  # noqa: E731
    return 1.5 * r(B, HQ, SQ, D), r(B, HK, SK, D), r(B, HK, SK, D), r(B, HQ, SQ, D)


def compare(pa, x, kw, fmt, out_dtype=None, kernel=0, mask=None):
    q, k, v, g = x
    f = [t.double().numpy() for t in x]
    add = None
    if mask is not None:
        add = mask.double().numpy() if mask.dtype == torch.float32 else np.where(mask.numpy() != 0, 0.0, -np.inf)
    y = torch.from_numpy(forward(*f[:3], kw, add)).to(q.dtype)
    tc = fmt != "f32" and q.shape[3] == 128 and kernel == 0 and mask is None
    want, err = gradient(f[0], f[1], f[2], y.double().numpy(), f[3], kw, U[fmt] if tc else 0.0,
                         2.0 ** -25 if tc and fmt == "f16" else 0.0, add)
    dev = {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in kw.items()}
    out = tuple(torch.full(t.shape, math.nan, dtype=out_dtype or q.dtype, device="cuda") for t in (q, k, k))
    got = pa.attention_vjp_scored(*(t.cuda() for t in (q, k, v, y, g)), None if mask is None else mask.cuda(), **dev,
                                  out_dtype=out_dtype, kernel=kernel, out=out)
    torch.cuda.synchronize()
    for name, a, w, e in zip(("dq", "dk", "dv"), got, want, err):
        o = a.double().cpu().numpy()
        half = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[a.dtype]
        lim = e + half * (np.abs(w) + e) + (2.0 ** -25 if a.dtype == torch.float16 else 2.0 ** -140)
        assert np.all(np.isfinite(o)), name
        assert np.all(np.abs(o - w) <= lim), (name, float(np.max(np.abs(o - w) / lim)))
    return got


# ------------------------------------------------------------------ CPU: refusals
A = 1 << 24


def call(pa, score=True, softcap=0.0, window=0, slopes=None, prefix=None, scale=0.1, HQ=4, **o):
    opts = pa.VjpOpts(dtype=2, out_dtype=-1, workspace=20 * A, workspace_bytes=1 << 30)
    for n, v in o.items():
        setattr(opts, n, v)
    s = pa.Score(softcap=softcap, window=window, slopes=slopes, prefix=prefix)
    p = [ctypes.c_void_p((i + 1) * A) for i in range(9)]
    p[5] = None
    return pa.LIB.pa_attention_vjp_scored(*p, ctypes.c_float(scale), 1, HQ, 2, 8, 8, 64, ctypes.byref(s) if score else None,
                                          ctypes.byref(opts), None)


@pytest.mark.parametrize("kw,code", [
    (dict(score=False), -1), (dict(softcap=-1.0), -2), (dict(softcap=math.nan), -2), (dict(softcap=math.inf), -2), (dict(softcap=1e-40), -2), (dict(window=-3), -2),
    (dict(slopes=A + 1), -4), (dict(prefix=A + 2), -4), (dict(scale=-1.0), -2), (dict(HQ=3), -2), (dict(dtype=9), -3),
    (dict(workspace=None), -1), (dict(workspace_bytes=4), -5), (dict(mask_kind=1), -1),
])
def test_refusals(pa, kw, code):
    assert call(pa, **kw) == code


# ------------------------------------------------------------------ GPU
SHAPES = [  # B, HQ, HK, SQ, SK
    (1, 1, 1, 1, 1), (2, 4, 2, 130, 130), (1, 6, 2, 300, 257), (2, 3, 1, 100, 400), (1, 2, 2, 513, 64),
]
MODS = [
    dict(softcap=20.0), dict(softcap=2.0), dict(slopes=True), dict(window=1), dict(window=100, prefix=40), dict(prefix=200),
    dict(softcap=10.0, slopes=True, window=150, prefix=33), dict(window=2 ** 31 - 1, prefix=-1),
]


def modified(mod, B, HQ, causal, D):
    kw = dict(scale=1 / math.sqrt(D), causal=causal, softcap=mod.get("softcap", 0.0), window=mod.get("window", 0))
    if mod.get("slopes"):
        kw["slopes"] = (2.0 ** (-8.0 * (torch.arange(HQ) + 1.0) / HQ)).float()
    if "prefix" in mod:
        kw["prefix"] = (torch.tensor([mod["prefix"]] * B) - 5 * torch.arange(B)).to(torch.int32)
    return kw


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_tensor_cores_match_64_bits(pa, shape, fmt):
    B, HQ, HK, SQ, SK = SHAPES[shape]
    x = make(shape, fmt, B, HQ, HK, SQ, SK, 128)
    for i, mod in enumerate(MODS):
        kw = modified(mod, B, HQ, (i + shape) % 2 == 0, 128)
        compare(pa, x, kw, fmt, torch.float32 if i % 2 else None)


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [0.3, 60.0, 75.0, 1e3, 1e6])
def test_caps_of_every_size(pa, cap):
    # a cap that saturates nearly all scores, both sides of the one that needs no
    # maximum, and one so large that it changes nothing
    x = make(15, "f16", 1, 2, 1, 200, 300, 128)
    for mod in (dict(softcap=cap), dict(softcap=cap, slopes=True, window=90)):
        compare(pa, x, modified(mod, 1, 2, False, 128), "f16", torch.float32)


@pytest.mark.gpu
def test_scores_on_both_sides_of_the_polynomial(pa):
    q, k, v, g = make(16, "bf16", 1, 2, 1, 300, 300, 128)
    q = torch.where(torch.rand(q.shape[2], 1, generator=torch.Generator().manual_seed(1)) < 0.3, 8 * q, q).to(q.dtype)
    compare(pa, (q, k, v, g), modified(dict(softcap=15.0), 1, 2, True, 128), "bf16", torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
def test_long_rows_windows_and_skipped_tiles(pa, causal):
    x = make(9, "bf16", 1, 2, 1, 1500, 1500, 128)
    for mod in (dict(window=130), dict(window=500, prefix=300), dict(window=64, prefix=1, softcap=50.0), dict(prefix=1490)):
        compare(pa, x, modified(mod, 1, 2, causal, 128), "bf16", torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,D", [("f32", 64), ("f32", 128), ("f16", 64), ("bf16", 40), ("f16", 128)])
def test_cuda_cores_match_64_bits(pa, fmt, D):
    for shape in (1, 3, 4):
        B, HQ, HK, SQ, SK = SHAPES[shape]
        x = make(20 + shape, fmt, B, HQ, HK, SQ, SK, D)
        for i, mod in enumerate(MODS):
            compare(pa, x, modified(mod, B, HQ, (i + shape) % 2 == 1, D), fmt, torch.float32, kernel=1)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bool", "add"])
def test_masks_add_to_the_modified_scores(pa, kind):
    x = make(31, "f32", 2, 4, 2, 40, 50, 64)
    g = torch.Generator().manual_seed(3)
    if kind == "bool":
        mask = (torch.rand(2, 1, 40, 50, generator=g) < 0.7).to(torch.uint8)
        mask[0, 0, 7] = 0  # a row that sees nothing
    else:
        mask = torch.randn(1, 4, 40, 50, generator=g)
        mask[0, 2, 9] = -math.inf
    for mod in (MODS[6], MODS[4]):
        compare(pa, x, modified(mod, 2, 4, True, 64), "f32", mask=mask)


@pytest.mark.gpu
def test_rows_without_keys_and_keys_without_rows(pa):
    # rows past SK + window see nothing; with a window keys past SQ are seen by no row
    for fmt in ("bf16", "f32"):
        x = make(40, fmt, 1, 2, 1, 300, 100, 128)
        got = compare(pa, x, modified(dict(window=20), 1, 2, True, 128), fmt)
        assert float(got[0][0, :, 119:].abs().max()) == 0.0
        x = make(41, fmt, 1, 2, 1, 100, 300, 128)
        got = compare(pa, x, modified(dict(window=20), 1, 2, False, 128), fmt)
        assert float(got[1][0, :, 119:].abs().max()) == 0.0 and float(got[2][0, :, 119:].abs().max()) == 0.0


@pytest.mark.gpu
def test_without_modification_equals_the_plain_gradient(pa):
    # one key tile a row: dq has a single term per element, so its reduction order cannot differ
    q, k, v, g = (t.cuda() for t in make(50, "bf16", 1, 4, 2, 200, 128, 128))
    y = q.clone()
    a = pa.attention_vjp(q, k, v, y, g, scale=0.09, causal=True)
    b = pa.attention_vjp_scored(q, k, v, y, g, scale=0.09, causal=True)
    for s, t in zip(a, b):
        # scores are scaled before or after the bias: one rounding of the exponent each
        assert torch.allclose(s.float(), t.float(), rtol=2.0 ** -7, atol=2.0 ** -7 * float(s.float().abs().max()))


@pytest.mark.gpu
def test_matches_differences_of_the_forward_pass(pa):
    # d/de <g, y(x + e d)> for random directions, central differences in 64 bits
    kw = modified(dict(softcap=6.0, slopes=True, window=30, prefix=5), 1, 4, True, 64)
    x = make(60, "f32", 1, 4, 2, 50, 50, 64)
    f = [t.double().numpy() for t in x]
    y = torch.from_numpy(forward(*f[:3], kw)).float()
    dev = {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in kw.items()}
    got = pa.attention_vjp_scored(*(t.cuda() for t in (*x[:3], y, x[3])), **dev)
    torch.cuda.synchronize()
    rng = np.random.default_rng(0)
    for n in range(3):
        d = rng.standard_normal(f[n].shape)
        e = 1e-5
        vals = []
        for s in (e, -e):
            z = list(f[:3])
            z[n] = f[n] + s * d
            vals.append((forward(*z, kw) * f[3]).sum())
        num = (vals[0] - vals[1]) / (2 * e)
        a = got[n].double().cpu().numpy()
        # float32 gradients: 2^-18 of the summed magnitudes; the difference's own error is of order e^2
        assert abs(num - (a * d).sum()) <= 2.0 ** -18 * (np.abs(a) * np.abs(d)).sum() + 1e-6


@pytest.mark.gpu
def test_graph_replay_and_another_stream(pa):
    q, k, v, g = (t.cuda() for t in make(70, "f16", 1, 4, 2, 200, 200, 128))
    pre = torch.tensor([9], dtype=torch.int32, device="cuda")
    plan = pa.ScoredVjpPlan(q, k, v, q, g, scale=0.09, causal=True, softcap=15.0, window=70, prefix=pre, out_dtype=torch.float32)
    plan.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
    q.mul_(0.5)
    pre.fill_(50)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (plan.dq, plan.dk, plan.dv)]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        plan.run()
    side.synchronize()
    assert torch.equal(got[1], plan.dk) and torch.equal(got[2], plan.dv)
    assert torch.allclose(got[0], plan.dq, rtol=1e-4, atol=1e-5)  # float32 reductions in another order


def test_workspace_sizes(pa):
    f, g = pa.LIB.pa_attention_vjp_scored_workspace_bytes, pa.LIB.pa_attention_vjp_workspace_bytes
    # few key tiles and grouped heads: partial dk and dv of every query head
    assert f(1, 4, 2, 200, 200, 128, 2, -1) == g(1, 4, 200, 128, 2, -1) + 2 * 4 * 200 * 128 * 4
    # no groups, no tensor cores, many tiles: nothing on top
    assert f(1, 4, 4, 200, 200, 128, 2, -1) == g(1, 4, 200, 128, 2, -1)
    assert f(1, 4, 2, 200, 200, 64, 2, -1) == g(1, 4, 200, 64, 2, -1)
    assert f(64, 32, 8, 2048, 2048, 128, 2, -1) == g(64, 32, 2048, 128, 2, -1)
    assert f(1, 4, 3, 200, 200, 128, 2, -1) == f(1, 4, 2, 200, 200, 128, 9, -1) == 0


@pytest.mark.gpu
def test_more_key_tiles_than_the_split_takes(pa):
    # 2 x 4 heads x 40 tiles: one CTA per group, no partial sums
    x = make(80, "f16", 2, 8, 4, 70, 5000, 128)
    compare(pa, x, modified(dict(softcap=12.0, prefix=700), 2, 8, False, 128), "f16", torch.float32)


@pytest.mark.gpu
def test_refused_arguments(pa):
    q, k, v, g = (t.cuda() for t in make(70, "f16", 1, 4, 2, 20, 20, 128))
    for bad in (dict(slopes=torch.zeros(5, device="cuda")), dict(prefix=torch.zeros(1, device="cuda")), dict(slopes=torch.zeros(4))):
        with pytest.raises(ValueError):
            pa.attention_vjp_scored(q, k, v, q, g, scale=0.1, **bad)
    with pytest.raises(pa.PagedAttentionError):
        pa.attention_vjp_scored(q, k, v, q, g, scale=0.1, window=-1)


@pytest.mark.gpu
@pytest.mark.parametrize("HK", [1, 4])
@pytest.mark.parametrize("SQ,SK", [(0, 130), (130, 0), (0, 0)])
def test_no_rows_or_no_keys(pa, SQ, SK, HK):
    # native outputs: the launch that rounds dq and joins the groups comes behind
    # the statistics alone, the backward alone, or nothing
    q, k, v, g = (t.cuda() for t in make(90, "bf16", 2, 4, HK, SQ, SK, 128))
    out = tuple(torch.full(t.shape, 3.0, dtype=torch.bfloat16, device="cuda") for t in (q, k, k))
    pa.attention_vjp_scored(q, k, v, q, g, scale=0.1, softcap=20.0, window=40, out=out)
    torch.cuda.synchronize()
    assert all(not t.any() for t in out)


@pytest.mark.gpu
def test_calls_back_to_back_on_other_inputs(pa):
    # launches that overlap their predecessor's end: calls of two shapes in turn, one
    # of them split by heads, and one plan whose inputs change between its calls
    kw = dict(scale=0.09, causal=True, softcap=30.0)
    sets = [[t.cuda() for t in make(100 + i, "bf16", 2, 8, 2, s, s, 128)] for i, s in enumerate((900, 900, 300))]
    plans = [pa.ScoredVjpPlan(q, k, v, q, g, **kw) for q, k, v, g in (sets[0], sets[2])]
    want = []
    for q, k, v, g in sets:
        want.append([t.clone() for t in pa.attention_vjp_scored(q, k, v, q, g, **kw)])
    torch.cuda.synchronize()
    live = [t.clone() for t in sets[0]]
    moving = pa.ScoredVjpPlan(live[0], live[1], live[2], live[0], live[3], **kw)
    got = []
    for n in range(12):
        for a, b in zip(live, sets[n % 2]):
            a.copy_(b)
        for plan in (moving, *plans):
            got.append((n, [t.clone() for t in plan.run()]))
    torch.cuda.synchronize()
    for i, (n, g) in enumerate(got):
        w = want[(n % 2, 0, 2)[i % 3]]
        assert torch.equal(g[1], w[1]) and torch.equal(g[2], w[2]), i
        # dq: sums in another order, then one rounding to bfloat16
        assert torch.allclose(g[0].float(), w[0].float(), rtol=2.0 ** -7, atol=1e-5), i


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,D,kernel", [("f32", 64, 0), ("f16", 64, 0), ("bf16", 128, 1), ("bf16", 128, 0), ("f16", 128, 0)])
def test_values_of_hidden_keys_may_be_anything(pa, fmt, D, kernel):
    # v of keys that no row sees holds infinities and NaN; both kernels give the gradient of finite ones
    B, HQ, HK, SQ, SK = 1, 4, 2, 90, 300
    q, k, v, g = make(120, fmt, B, HQ, HK, SQ, SK, D)
    tc = D == 128 and kernel == 0
    for kw, first in ((modified(dict(window=20), B, HQ, False, D), SQ + 19), (modified(dict(softcap=9.0, slopes=True), B, HQ, True, D), SQ)):
        dead = torch.arange(SK) >= first
        bad = v.clone()
        bad[:, :, first::3], bad[:, :, first + 1::3], bad[:, :, first + 2::3] = math.nan, math.inf, -math.inf
        f = [t.double().numpy() for t in (q, k, v, g)]
        y = torch.from_numpy(forward(*f[:3], kw)).to(q.dtype)
        want, err = gradient(*f[:3], y.double().numpy(), f[3], kw, U[fmt] if tc else 0.0, 2.0 ** -25 if tc and fmt == "f16" else 0.0)
        dev = {n: (t.cuda() if isinstance(t, torch.Tensor) else t) for n, t in kw.items()}
        got = pa.attention_vjp_scored(*(t.cuda() for t in (q, k, bad, y, g)), **dev, out_dtype=torch.float32, kernel=kernel)
        torch.cuda.synchronize()
        for name, a, w, e in zip(("dq", "dk", "dv"), got, want, err):
            o = a.double().cpu().numpy()
            assert np.all(np.abs(o - w) <= e + 2.0 ** -24 * (np.abs(w) + e) + 2.0 ** -140), name
        assert not got[1][:, :, dead].any() and not got[2][:, :, dead].any()


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("kind", ["causal", "bool", "add"])
def test_values_hidden_from_the_plain_gradient_may_be_anything(pa, kind, kernel):
    # the same of pa_attention_vjp: the causal rule, and masks (which run on the CUDA cores)
    q, k, v, g = (t.cuda() for t in make(121, "f32" if kind != "causal" else "f16", 1, 4, 2, 60, 130, 128))
    hidden, mask = torch.arange(130) >= 60, None
    if kind != "causal":
        mask = (~hidden).to(torch.uint8).view(1, 1, 1, 130).expand(1, 1, 60, 130).contiguous()
        if kind == "add":
            mask = torch.where(mask != 0, 0.0, -math.inf).float()
        mask = mask.cuda()
    y, bad = q.clone(), v.clone()
    bad[:, :, 60::2], bad[:, :, 61::2] = math.nan, math.inf
    call = lambda x: pa.attention_vjp(q, k, x, y, g, mask, scale=0.09, causal=kind == "causal", kernel=kernel,  # noqa: E731
                                      out_dtype=torch.float32)
    want, got = call(v), call(bad)
    assert all(torch.isfinite(t).all() for t in got)
    assert torch.equal(want[1], got[1]) and torch.equal(want[2], got[2])
    # dq: the 60 visible keys are four tiles of 16 (CUDA cores) whose parts are added in any order: each
    # order is off by at most 3 roundings of the sum of the parts' magnitudes, which is at most |ds| |k|
    Q, K, V, G = (t.double().repeat_interleave(4 // t.shape[1], 1) for t in (q, k, v, g))
    seen = ~hidden.cuda() & ((torch.arange(130) <= torch.arange(60)[:, None]).cuda() | (kind != "causal"))
    p = torch.softmax((0.09 * Q @ K.mT).masked_fill(~seen, -math.inf), -1)
    ds = 0.09 * p * (G @ V.mT - (Q * G).sum(-1, keepdim=True))
    assert torch.all((want[0] - got[0]).abs() <= 2 * 3 * 2.0 ** -24 * 1.01 * (ds.abs() @ K.abs()))


@pytest.mark.parametrize("softcap,scale", [(3e38, 0.1), (2.4e38, 1e10), (1e37, 0.1), (2e31, 0.1), (1e-32, 0.1), (1e-45, 0.1), (1.0, 1e-31)])
def test_refused_caps(pa, softcap, scale):
    assert call(pa, softcap=softcap, scale=scale) == -2


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,D", [("f16", 128), ("f32", 64)])
@pytest.mark.parametrize("cap", [1e20, 1e29])
def test_caps_that_change_nothing(pa, fmt, D, cap):
    x = make(17, fmt, 1, 2, 1, 150, 200, D)
    for mod in (dict(softcap=cap), dict(softcap=cap, slopes=True, window=90)):
        compare(pa, x, modified(mod, 1, 2, False, D), fmt, torch.float32)
