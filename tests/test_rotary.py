"""Rotary positions (include/pa_rotary.h): the frequency table and the
refusals on the CPU, the kernels against 64-bit arithmetic on the GPU.

Error bound of one rotated element: factor * (|u| + |v|) * 2^-21 plus half a
step of the dtype at the result.  The reduced angle's float conversion is off
by 2^-24 of at most pi / 4 and its truncation to 2^-32 turns by 2^-29 radians;
sincospi adds at most 2 units in the last place of values below 1 (2^-23),
the factor's product 2^-24: together less than 2^-22 on cosine and sine.  The
two products and their sum round three times by 2^-24 of |u| + |v|.
"""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

STEP = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # f32: in the bound already
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SCALINGS = [None, ("linear", 4.0), ("ntk", 8.0), ("bands", 8.0, 4096, 1.0, 4.0), ("yarn", 16.0, 2048, 32.0, 1.0)]


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_182_gb300 import _build

    _build.build()
    from paged_kv_cache_182_gb300 import binding

    return binding


# ------------------------------------------------------------------ reference
def turned(x, pos, inv, factor, interleaved, inverse=False):
    """x float64 [B, H, N, D] turned by pos [B, N]; and |u| + |v| per element."""
    half = len(inv)
    ang = pos.astype(np.longdouble)[:, None, :, None] * np.array(inv, dtype=np.longdouble)
    ang = np.remainder(ang, 2 * np.longdouble(math.pi) + np.longdouble(1.2246467991473532e-16) * 2)
    c, s = np.cos(ang.astype(np.float64)), np.sin(ang.astype(np.float64))
    if inverse:
        s = -s
    y, mag = x.copy(), np.abs(x)
    iu = np.arange(half) * 2 if interleaved else np.arange(half)
    iv = iu + 1 if interleaved else iu + half
    u, v = x[..., iu], x[..., iv]
    y[..., iu], y[..., iv] = factor * (u * c - v * s), factor * (u * s + v * c)
    mag[..., iu] = mag[..., iv] = factor * (np.abs(u) + np.abs(v))
    return y, mag


def check(got, want, mag, fmt, rot):
    g = got.detach().cpu().double().numpy()
    bound = mag * 2.0 ** -21 + STEP[fmt] * np.abs(want) * 1.001 + (2.0 ** -25 if fmt == "f16" else 0.0)
    bound[..., rot:] = 0.0
    assert np.all(np.abs(g - want) <= bound), float(np.max(np.abs(g - want) - bound))


# ------------------------------------------------------------------ CPU: table
@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("rot", [4, 10, 64, 128])
def test_table_is_the_frequency_in_turns(pa, rot, scaling):
    inv, factor = pa.rotary_frequencies(rot, base=500000.0, scaling=scaling)
    t = pa.rotary_table(rot, base=500000.0, scaling=scaling, device="cpu")
    assert t.rot == rot and t.factor == factor and tuple(t.turns.shape) == (rot // 2,)
    for x, w in zip(inv, t.turns.tolist()):
        assert abs(Fraction(w % 2 ** 64, 2 ** 64) * 2 * Fraction(math.pi) - Fraction(x)) < Fraction(x) / 10 ** 15 + Fraction(1, 2 ** 62)


def test_scalings_leave_fast_pairs_and_stretch_slow_ones(pa):
    plain, _ = pa.rotary_frequencies(128)
    for scaling in (("bands", 8.0, 4096, 1.0, 4.0), ("yarn", 8.0, 4096, 32.0, 1.0)):
        inv, factor = pa.rotary_frequencies(128, scaling=scaling)
        assert inv[0] == plain[0] and math.isclose(inv[-1], plain[-1] / 8.0, rel_tol=1e-12)
        assert all(a <= b and a >= b / 8.0 - 1e-18 for a, b in zip(inv, plain))
        assert (factor > 1.0) == (scaling[0] == "yarn")
    ntk, _ = pa.rotary_frequencies(128, scaling=("ntk", 8.0))
    assert ntk[0] == plain[0] and math.isclose(ntk[-1], plain[-1] / 8.0, rel_tol=1e-12)


@pytest.mark.parametrize("bad", [dict(rot=3), dict(rot=0), dict(rot=8, base=1.0), dict(rot=8, scaling=("linear",)),
                                 dict(rot=8, scaling=("linear", -1.0)), dict(rot=8, scaling=("other", 1.0)),
                                 dict(rot=2, scaling=("ntk", 2.0)), dict(rot=8, scaling=("bands", 2.0, 128, 4.0, 4.0))])
def test_table_refusals(pa, bad):
    rot = bad.pop("rot")
    with pytest.raises(ValueError):
        pa.rotary_table(rot, device="cpu", **bad)


# ------------------------------------------------------------------ CPU: refusals
A = 1 << 20  # an aligned address that is never read


def call(pa, B=2, H=4, KV=2, N=3, D=64, rot=32, dtype=1, q=A, k=2 * A, pos=3 * A, tab=4 * A, qo=5 * A, ko=6 * A,
         factor=1.0, strides=None, store=False, nopts=False, **o):
    opts = pa.RotaryOpts(dtype=dtype, factor=factor)
    for name, heads in (("q_strides", H), ("k_strides", KV), ("v_strides", KV)):
        getattr(opts, name)[:] = (heads * N * D, N * D, D) if strides is None else strides
    if store:
        opts.slot_mapping, opts.v, opts.k_cache, opts.v_cache = 7 * A, 8 * A, 9 * A, 10 * A
        opts.BLOCK, opts.num_blocks = 16, 4
    for name, v in o.items():
        setattr(opts, name, v)
    p = lambda x: None if x is None else ctypes.c_void_p(x)  # noqa: E731
    return pa.LIB.pa_rotary(p(q), p(k), p(pos), p(tab), p(qo), p(ko), B, H, KV, N, D, rot,
                            None if nopts else ctypes.byref(opts), None)


NULL, DIMS, UNSUP, ALIGN = -1, -2, -3, -4


@pytest.mark.parametrize("kw,code", [
    (dict(nopts=True), NULL), (dict(q=None), NULL), (dict(k=None), NULL), (dict(pos=None), NULL), (dict(tab=None), NULL),
    (dict(qo=None), NULL), (dict(ko=None), NULL), (dict(store=True, v=None), NULL), (dict(store=True, k_cache=None), NULL),
    (dict(B=-1), DIMS), (dict(H=0, KV=0), DIMS), (dict(rot=33), DIMS), (dict(rot=0), DIMS), (dict(rot=66), DIMS),
    (dict(factor=math.nan), DIMS), (dict(N=-1), DIMS), (dict(B=1 << 16, N=1 << 15), DIMS), (dict(store=True, BLOCK=0), DIMS),
    (dict(store=True, num_blocks=1 << 28, BLOCK=16), DIMS),
    (dict(qo=A), DIMS), (dict(qo=A + 64), DIMS), (dict(ko=5 * A), DIMS), (dict(store=True, k_cache=8 * A), DIMS),
    (dict(store=True, k_cache=10 * A), DIMS),
    (dict(dtype=3), UNSUP), (dict(D=68, rot=4), UNSUP), (dict(D=2048, rot=4), UNSUP), (dict(store=True, N=65537), UNSUP),
    (dict(q=A + 8), ALIGN), (dict(ko=6 * A + 2), ALIGN), (dict(pos=3 * A + 2), ALIGN), (dict(tab=4 * A + 4), ALIGN),
    (dict(strides=(768, 196, 64)), ALIGN), (dict(strides=(768, 192, -64)), ALIGN), (dict(strides=(1 << 41, 192, 64)), DIMS),
    (dict(store=True, v_cache=10 * A + 8), ALIGN),
])
def test_refusals(pa, kw, code):
    assert call(pa, **kw) == code


def test_nothing_to_do(pa):
    assert call(pa, B=0, q=None) == 0
    assert call(pa, N=0, q=None) == 0


# ------------------------------------------------------------------ GPU
def make(seed, fmt, B, H, KV, N, D, far, fused, dev="cuda"):
    g = torch.Generator().manual_seed(seed)
    rows = torch.randn(B, N, H + 2 * KV, D, generator=g).to(DT[fmt]).to(dev).transpose(1, 2)
    q, k, v = rows[:, :H], rows[:, H:H + KV], rows[:, H + KV:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, far, (B, N), generator=g, dtype=torch.int32).to(dev)
    return q, k, v, pos


CASES = [  # B, H, KV, N, D, rot, far
    (1, 1, 1, 1, 64, 64, 10), (2, 4, 2, 3, 64, 32, 5000), (3, 5, 1, 17, 128, 128, 1 << 20), (1, 8, 8, 1, 256, 256, 2 ** 31 - 1),
    (2, 3, 3, 33, 80, 40, 100000), (1, 2, 1, 300, 72, 2, 1 << 16), (4, 7, 1, 5, 96, 50, 1 << 20), (1, 12, 4, 129, 128, 36, 4096),
    (65, 2, 2, 2, 64, 62, 1 << 18), (1, 1, 1, 3, 1024, 1024, 1 << 20),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_matches_64_bits(pa, case, interleaved, fmt):
    B, H, KV, N, D, rot, far = case
    scaling = SCALINGS[(B + N + rot) % len(SCALINGS)] if rot >= 4 else None
    q, k, _, pos = make(sum(case), fmt, B, H, KV, N, D, far, fused=N % 2 == 1)
    table = pa.rotary_table(rot, scaling=scaling)
    inv, factor = pa.rotary_frequencies(rot, scaling=scaling)
    for inverse in (False, True):
        qo, ko = pa.rotary(q, k, pos, table, interleaved=interleaved, inverse=inverse)
        torch.cuda.synchronize()
        for x, y in ((q, qo), (k, ko)):
            check(y, *turned(x.double().cpu().numpy(), pos.cpu().numpy(), inv, factor, interleaved, inverse), fmt, rot)


@pytest.mark.gpu
def test_one_tensor_alone_and_negative_positions(pa):
    q, k, _, pos = make(5, "f32", 2, 3, 2, 4, 64, 1000, False)
    table = pa.rotary_table(64)
    inv, _ = pa.rotary_frequencies(64)
    both = pa.rotary(q, k, pos, table)
    alone = pa.rotary(q, None, pos, table)
    assert alone[1] is None and torch.equal(alone[0], both[0])
    assert torch.equal(pa.rotary(None, k, pos, table)[1], both[1])
    back = pa.rotary(q, None, -pos, table)[0]
    check(back, *turned(q.double().cpu().numpy(), -pos.cpu().numpy(), inv, 1.0, False), "f32", 64)
    # a turn by -p is the inverse turn by p, to the bit
    assert torch.equal(back, pa.rotary(q, None, pos, table, inverse=True)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_is_the_transpose_and_matches_differences(pa, interleaved):
    q, k, _, pos = make(7, "f32", 2, 3, 1, 5, 64, 100000, True)
    table = pa.rotary_table(24, scaling=("yarn", 4.0, 512, 32.0, 1.0))
    g = torch.randn(2, 3, 5, 64, generator=torch.Generator().manual_seed(1)).cuda()
    dx = pa.rotary(g, None, pos, table, interleaved=interleaved, inverse=True)[0]
    # d/dt <g, R(q + t h)> = <R^T g, h>: R is linear, so a difference of any
    # length is exact up to the rounding of R's values (2^-21 of them each)
    h = torch.randn(q.shape, generator=torch.Generator().manual_seed(2)).cuda()
    plus = pa.rotary(q + h, None, pos, table, interleaved=interleaved)[0].double()
    minus = pa.rotary(q - h, None, pos, table, interleaved=interleaved)[0].double()
    num = ((plus - minus) * g.double()).sum() / 2
    ana = (dx.double() * h.double()).sum()
    size = float((g.double().abs() * (plus.abs() + minus.abs() + 1)).sum())
    assert abs(float(num - ana)) <= size * 2.0 ** -19


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N", [1, 4])
def test_append_stores_rotated_keys_and_values(pa, N, fmt):
    B, H, KV, D, BLOCK, NB = 5, 6, 3, 64, 16, 7
    q, k, v, pos = make(11 + N, fmt, B, H, KV, N, D, 70000, True)
    kc = torch.full((NB, BLOCK, KV, D), 9.0, dtype=DT[fmt], device="cuda")
    vc = torch.full_like(kc, 8.0)
    slots = torch.randperm(NB * BLOCK, generator=torch.Generator().manual_seed(3))[: B * N].view(B, N).to(torch.int32)
    slots[1, 0] = -1
    if N > 1:
        slots[2, 1] = slots[2, 3]  # the later row wins
    slots[4, 0] = NB * BLOCK  # outside the pool
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = pa.rotary_table(D)
    qo, ko = pa.rotary_append(q, k, v, pos, slots.cuda(), kc, vc, table, status=status)
    plain = pa.rotary(q, k, pos, table)
    assert torch.equal(qo, plain[0]) and torch.equal(ko, plain[1])
    wk, wv = torch.full_like(kc, 9.0).view(-1, KV, D), torch.full_like(vc, 8.0).view(-1, KV, D)
    for b in range(B):
        for n in range(N):
            s = int(slots[b, n])
            if 0 <= s < NB * BLOCK:
                wk[s], wv[s] = ko[b, :, n], v[b, :, n]
    assert torch.equal(kc.view(-1, KV, D), wk) and torch.equal(vc.view(-1, KV, D), wv)
    assert int(status) == pa.PA_STATUS_BAD_SLOT


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,D,H,KV", [("bf16", 64, 4, 2), ("f32", 128, 0, 3), ("f16", 64, 40, 8)])
def test_append_of_a_long_prompt_with_repeated_slots(pa, fmt, D, H, KV):
    B, N, BLOCK, NB = 2, 300, 16, 8  # 128 slots a sequence: rows come round more than twice
    q, k, v, pos = make(31, fmt, B, max(H, 1), KV, N, D, 70000, True)
    kc = torch.zeros((2 * NB, BLOCK, KV, D), dtype=DT[fmt], device="cuda")
    vc = torch.zeros_like(kc)
    slots = (torch.arange(N) % 128 + 128 * torch.arange(B).view(-1, 1)).to(torch.int32)
    slots[0, 250:] = -1
    table = pa.rotary_table(D)
    _, ko = pa.rotary_append(q if H else None, k, v, pos, slots.cuda(), kc, vc, table)
    wk, wv = torch.zeros_like(kc).view(-1, KV, D), torch.zeros_like(vc).view(-1, KV, D)
    for b in range(B):
        for n in range(N):
            if slots[b, n] >= 0:
                wk[slots[b, n]], wv[slots[b, n]] = ko[b, :, n], v[b, :, n]
    assert torch.equal(kc.view(-1, KV, D), wk) and torch.equal(vc.view(-1, KV, D), wv)


@pytest.mark.gpu
def test_graph_replay_other_stream_and_refused_arguments(pa):
    q, k, v, pos = make(21, "f16", 3, 4, 2, 2, 64, 5000, False)
    table = pa.rotary_table(64)
    want = [t.clone() for t in pa.rotary(q, k, pos, table)]
    plan = pa.RotaryPlan(q, k, pos, table)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        plan.run()
    side.synchronize()
    assert torch.equal(plan.q_out, want[0]) and torch.equal(plan.k_out, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.run()
    pos.add_(7)
    want = [t.clone() for t in pa.rotary(q, k, pos, table)]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(plan.q_out, want[0]) and torch.equal(plan.k_out, want[1])
    with pytest.raises(pa.PagedAttentionError):
        pa.RotaryPlan(q, None, pos, table, q_out=q).run()
    with pytest.raises(ValueError):
        pa.RotaryPlan(q, k, pos.long(), table)
    with pytest.raises(ValueError):
        pa.RotaryPlan(q.transpose(2, 3), None, pos, table)
    with pytest.raises(TypeError):
        pa.RotaryPlan(q, k.float(), pos, table)
    with pytest.raises(ValueError):
        three = torch.zeros(4, 16, 3, 64, dtype=k.dtype, device="cuda")  # k has two heads
        pa.RotaryAppendPlan(q, k, v, pos, pos, three, three.clone(), table)
