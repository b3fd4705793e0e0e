"""The operators as they are used together: a serving loop (rotate and store the
new rows, decode with modified scores and key weights, evict when over budget,
go on) and a training step (rotate, attend, gradient, rotate back), each
against 64-bit arithmetic; and the loop's step captured in one graph.

Bound of a decode output in the loop (float32): a rotated element is off by
2^-21 of its pair, so a score by delta <= scale sum |q k| (2^-20 + D 2^-23) +
2^-21 |t|; a softmax average by at most 4 delta max |v| (twice the first-order
2 delta), plus 2^-20 max |v| for weights, sums and the value rows' products.
"""
import math

import numpy as np
import pytest
import torch

from test_evict import kept_of
from test_rotary import turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_182_gb300 import binding

    return binding


class Loop:
    """Device state of a serving loop and the calls of one step."""

    def __init__(self, pa, lens, budget, dtype=torch.float32, H=4, KV=2, D=64, BLOCK=16):
        self.pa, self.B, self.H, self.KV, self.D, self.BLOCK, self.budget = pa, len(lens), H, KV, D, BLOCK, budget
        g = torch.Generator().manual_seed(3)
        blocks = 8
        perm = torch.randperm(self.B * blocks, generator=g).to(torch.int32)
        self.table = perm.view(self.B, blocks).contiguous().cuda()
        self.kc = torch.randn(self.B * blocks, BLOCK, KV, D, generator=g).to(dtype).cuda()
        self.vc = torch.randn(self.B * blocks, BLOCK, KV, D, generator=g).to(dtype).cuda()
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.pos = torch.tensor([[1000 + n] for n in lens], dtype=torch.int32, device="cuda")
        self.weights = torch.zeros(self.B, blocks * BLOCK, device="cuda")
        self.q = torch.zeros(self.B, H, 1, D, dtype=dtype, device="cuda")
        self.k, self.v = (torch.zeros(self.B, KV, 1, D, dtype=dtype, device="cuda") for _ in range(2))
        self.slopes = torch.tensor([0.5, 0.25, 0.125, 0.0625], device="cuda")
        self.prefix = torch.tensor([3] * self.B, dtype=torch.int32, device="cuda")
        self.rot = pa.rotary_table(D, scaling=("linear", 2.0))
        self.slots = torch.zeros(self.B, 1, dtype=torch.int32, device="cuda")
        self.turn = pa.RotaryAppendPlan(self.q, self.k, self.v, self.pos, self.slots, self.kc, self.vc, self.rot)
        self.scale = D ** -0.5
        self.attend = pa.ScoredPlan(self.turn.q_out, self.kc, self.vc, self.table, self.lens, self.turn.k_out, self.v,
                                    scale=self.scale, causal=True, softcap=8.0, slopes=self.slopes, window=30, prefix=self.prefix,
                                    key_weights=self.weights, decay=0.9)
        self.evict = pa.EvictPlan(self.kc, self.vc, self.table, self.lens, self.weights, budget=budget, keep_first=3, keep_last=8)

    def slot_of_next(self):
        at = self.lens.long().unsqueeze(1)
        self.slots.copy_(torch.gather(self.table, 1, at // self.BLOCK) * self.BLOCK + (at % self.BLOCK).to(torch.int32))

    def step(self):
        """One token of every sequence; every call is asynchronous on the current stream."""
        self.slot_of_next()
        self.turn.run()
        out, _ = self.attend.run()
        self.lens.add_(1)
        self.pos.add_(1)
        new, kept, weights = self.evict.run()
        self.lens.copy_(new)
        self.weights.copy_(weights)
        return out


def rows_of(loop, b, n):
    j = np.arange(n)
    slots = loop.table[b].cpu().numpy()[j // loop.BLOCK].astype(np.int64) * loop.BLOCK + j % loop.BLOCK
    return [x.double().cpu().numpy().reshape(-1, loop.KV, loop.D)[slots] for x in (loop.kc, loop.vc)]


def test_serving_loop_over_its_budget(pa):
    loop = Loop(pa, [38, 45, 20], 40)
    B, H, KV, D = loop.B, loop.H, loop.KV, loop.D
    G = H // KV
    inv, factor = pa.rotary_frequencies(D, scaling=("linear", 2.0))
    cache = [rows_of(loop, b, n) for b, n in enumerate(loop.lens.tolist())]  # what each sequence holds
    weights = [np.zeros(n) for n in loop.lens.tolist()]
    g = torch.Generator().manual_seed(8)
    for t in range(30):
        for x in (loop.q, loop.k, loop.v):
            x.copy_(torch.randn(x.shape, generator=g))
        pos = loop.pos.cpu().numpy()
        q, k, v = (x.double().cpu().numpy() for x in (loop.q, loop.k, loop.v))
        lens, before = loop.lens.tolist(), loop.weights.clone()
        out = loop.step()
        torch.cuda.synchronize()
        out = out.double().cpu().numpy()
        qr, _ = turned(q, pos, inv, factor, False)
        kr, _ = turned(k, pos, inv, factor, False)
        kept, new = loop.evict.kept.cpu().numpy(), loop.lens.tolist()
        wout = loop.weights.cpu().numpy()
        for b in range(B):
            n = lens[b]
            K = np.concatenate((cache[b][0], kr[b].transpose(1, 0, 2)))
            V = np.concatenate((cache[b][1], v[b].transpose(1, 0, 2)))
            j = np.arange(n + 1)
            seen = (j < 3) | (n - j < 30)
            w = np.concatenate((0.9 * weights[b], [0.0]))
            for h in range(H):
                kh = h // G
                dots = K[:, kh] @ qr[b, h, 0]
                mag = loop.scale * (np.abs(K[:, kh]) @ np.abs(qr[b, h, 0])) * (2.0 ** -20 + D * 2.0 ** -23)
                s = np.where(seen, 8 * np.tanh(loop.scale * dots / 8) - float(loop.slopes[h]) * (n - j), -np.inf)
                p = np.exp(s - s.max())
                p /= p.sum()
                w += p
                vmax = np.abs(V[:, kh]).max()
                delta = (mag + 2.0 ** -21 * np.abs(np.where(seen, s, 0))).max()
                assert np.all(np.abs(out[b, h, 0] - p @ V[:, kh]) <= 4 * delta * vmax + 2.0 ** -20 * vmax), (t, b, h)
            # the eviction goes by the weights that the decode kept (float32, close to these)
            m = min(n + 1, 40)
            ids = kept[b][:m]
            assert new[b] == m and np.all(kept[b][m:] == -1)
            # weights: p is off by at most 2 delta of itself, and 2^-20; delta below 2^-14 here
            assert np.all(np.abs(wout[b, :m] - w[ids]) <= (w[ids] + 1e-6) * 2.0 ** -12)
            assert np.all(wout[b, m:] == 0)
            gap = np.sort(w[3:n + 1 - 8])  # unless two weights nearly tie, the choice is that of 64 bits
            if n + 1 > 40 and np.diff(gap).min() > 1e-6 * gap.max() + 2.0 ** -12 * gap.max():
                assert list(ids) == kept_of(w, n + 1, 40, 3, 8), (t, b)
            cache[b] = [K[ids], V[ids]]
            weights[b] = wout[b, :m].astype(np.float64)
            K2, V2 = rows_of(loop, b, m)
            assert np.array_equal(V2, V[ids])
            assert np.all(np.abs(K2 - K[ids]) <= 2.0 ** -20 * (np.abs(K[ids]) + 4))
            cache[b][0] = K2  # as stored
        assert before.shape == loop.weights.shape
    assert loop.lens.tolist() == [40, 40, 40]


def test_the_loop_in_one_graph(pa):
    """Ten replays of a captured step equal ten eager steps, to the bit."""
    a, b = Loop(pa, [38, 45, 20], 40, torch.bfloat16), Loop(pa, [38, 45, 20], 40, torch.bfloat16)
    g = torch.Generator().manual_seed(9)
    steps = [[torch.randn(x.shape, generator=g).to(x.dtype).cuda() for x in (a.q, a.k, a.v)] for _ in range(10)]
    # capture without running: the state that the warm-up changed is put back
    keep = [x.clone() for x in (b.kc, b.vc, b.lens, b.pos, b.weights)]
    b.step()
    for x, y in zip((b.kc, b.vc, b.lens, b.pos, b.weights), keep):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.step()
    for new in steps:
        for loop in (a, b):
            for x, y in zip((loop.q, loop.k, loop.v), new):
                x.copy_(y)
        want = a.step().clone()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, out)
        for x, y in ((a.kc, b.kc), (a.vc, b.vc), (a.lens, b.lens), (a.weights, b.weights), (a.evict.kept, b.evict.kept)):
            assert torch.equal(x, y)


def test_training_step(pa):
    """Rotation, attention with modified scores, its gradient, the rotation back:
    against automatic differentiation of the whole in 64 bits.  Bound: 2e-5 of
    each gradient's largest value, the float32 backward's own."""
    B, H, KV, S, D = 2, 4, 2, 60, 64
    g = torch.Generator().manual_seed(5)
    q, k, v, grad = (torch.randn(B, n, S, D, generator=g) for n in (H, KV, KV, H))
    pos = (torch.arange(S, dtype=torch.int32) + 500).expand(B, S).contiguous()
    table = pa.rotary_table(48, scaling=("yarn", 4.0, 256, 32.0, 1.0))
    inv, factor = pa.rotary_frequencies(48, scaling=("yarn", 4.0, 256, 32.0, 1.0))
    slopes = torch.tensor([0.3, 0.1, 0.03, 0.01])
    prefix = torch.tensor([4, 0], dtype=torch.int32)
    cap, window, scale = 5.0, 25, D ** -0.5

    def rotate(x):
        a = pos.double()[:, None, :, None] * torch.tensor(inv, dtype=torch.float64)
        c, s = a.cos() * factor, a.sin() * factor
        u, w = x[..., :24], x[..., 24:48]
        return torch.cat((u * c - w * s, u * s + w * c, x[..., 48:]), -1)

    leaf = [x.double().requires_grad_() for x in (q, k, v)]
    Q, K, V = rotate(leaf[0]), rotate(leaf[1]).repeat_interleave(2, 1), leaf[2].repeat_interleave(2, 1)
    i, j = torch.arange(S).view(-1, 1), torch.arange(S).view(1, -1)
    t = cap * torch.tanh(scale * Q @ K.transpose(-1, -2) / cap) - slopes.double().view(1, -1, 1, 1) * (i - j).abs()
    seen = ((j <= i) & ((i - j).abs() < window)).view(1, 1, S, S) | (j.view(1, 1, 1, S) < prefix.view(-1, 1, 1, 1))
    y = torch.softmax(t.masked_fill(~seen, -math.inf), -1) @ V
    (y * grad.double()).sum().backward()

    qd, kd, vd, gd = (x.cuda() for x in (q, k, v, grad))
    qr, kr = pa.rotary(qd, kd, pos.cuda(), table)
    dq, dk, dv = pa.attention_vjp_scored(qr, kr, vd, y.detach().float().cuda(), gd, scale=scale, causal=True, softcap=cap,
                                         slopes=slopes.cuda(), window=window, prefix=prefix.cuda())
    dq, dk = pa.rotary(dq, dk, pos.cuda(), table, inverse=True)
    torch.cuda.synchronize()
    for name, a, x in (("dq", dq, leaf[0]), ("dk", dk, leaf[1]), ("dv", dv, leaf[2])):
        want = x.grad
        assert float((a.double().cpu() - want).abs().max()) <= 2e-5 * max(1.0, float(want.abs().max())), name


def test_two_loops_and_a_gradient_on_streams_of_their_own(pa):
    # every plan has its own workspace and scratch: what runs beside it changes nothing
    def state():
        loops = [Loop(pa, lens, 60, dtype=torch.float16, D=128) for lens in ([100, 75, 61, 20] * 6, [90, 118] * 4)]
        g = torch.Generator().manual_seed(21)
        x = [torch.randn(1, h, 700, 128, generator=g).half().cuda() for h in (4, 2, 2, 4)]
        grad = pa.ScoredVjpPlan(x[0], x[1], x[2], x[0], x[3], scale=0.09, causal=True, softcap=20.0, window=300)
        steps = [[torch.randn(t.shape, generator=g).half().cuda() for _ in range(12) for t in (loop.q, loop.k, loop.v)] for loop in loops]
        return loops, grad, steps

    def step(loop, rows, n):
        for t, r in zip((loop.q, loop.k, loop.v), rows[3 * n:3 * n + 3]):
            t.copy_(r)
        return loop.step().clone()

    loops, grad, rows = state()
    want = [[step(loop, r, n) for n in range(12)] for loop, r in zip(loops, rows)]
    want_end = [(loop.lens.clone(), loop.weights.clone(), loop.kc.clone()) for loop in loops]
    _, dk, dv = (t.clone() for t in grad.run())
    torch.cuda.synchronize()
    loops, grad, rows = state()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got, parts = [[], []], []
    for n in range(12):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(step(loops[i], rows[i], n))
        with torch.cuda.stream(streams[2]):
            parts.append([t.clone() for t in grad.run()[1:]])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(want[i], got[i]))
        assert all(torch.equal(a, b) for a, b in zip(want_end[i], (loops[i].lens, loops[i].weights, loops[i].kc)))
    assert all(torch.equal(a, dk) and torch.equal(b, dv) for a, b in parts)
