"""One-call functions given a stream that is not torch's current one: what
such a call allocates (and zero-fills) for itself belongs to the current
stream, so the given stream has to wait for that one before the launch, and
the memory may not be handed out again before the given stream has passed the
call.  The order of the calls is checked on the CPU with stand-ins for the
plans and streams, the results on the GPU while the current stream is busy."""
import contextlib
import math
import types

import pytest
import torch


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_182_gb300 import _build

    _build.build()
    from paged_kv_cache_182_gb300 import binding

    return binding


# ------------------------------------------------------------------ CPU: the order of the calls
class FakeStream:
    cuda_stream = 77

    def __init__(self, log, name):
        self.log, self.name = log, name

    def wait_stream(self, other):
        self.log.append(f"{self.name} waits for {other.name}")

    def synchronize(self):
        self.log.append(f"synchronize {self.name}")


class FakeTensor:
    def __init__(self, log, name):
        self.log, self.name = log, name

    def record_stream(self, stream):
        self.log.append(f"{self.name} kept for {stream.name}")


def fake_plan(log):
    class Fake:
        """Stands for every plan class: logs its construction and its launch."""

        shape = dict(B=2, H=4, KV=2, D=64, BLOCK=16, NQ=1, num_blocks=4, max_blocks=2)

        def __init__(self, *args, **kw):
            log.append("made")
            self.device = torch.device("cuda", 0)
            self._args = [0] * 20
            for name in ("out", "workspace", "scratch", "mask", "dq", "dk", "dv", "q_out", "k_out", "new_lens", "kept", "weights_out"):
                setattr(self, name, FakeTensor(log, name))

        def run(self, *args):
            log.append(f"run on {args[-1] and args[-1].name}")

    return Fake


CALLS = {  # function -> the plan class it makes, its positional arguments, what it allocates
    "decode": ("Plan", 7, ("out", "workspace")),
    "prefill": ("PrefillPlan", 7, ("out", "workspace")),
    "attention_vjp": ("VjpPlan", 5, ("dq", "dk", "dv", "workspace", "mask")),
    "decode_scored": ("ScoredPlan", 7, ("out", "workspace", "scratch")),
    "attention_vjp_scored": ("ScoredVjpPlan", 5, ("dq", "dk", "dv", "workspace", "mask")),
    "rotary": ("RotaryPlan", 4, ("q_out", "k_out")),
    "rotary_append": ("RotaryAppendPlan", 8, ("q_out", "k_out")),
    "cache_evict": ("EvictPlan", 5, ("new_lens", "kept", "weights_out")),
}


def keywords(name):
    return {"rotary": {}, "rotary_append": {}, "cache_evict": dict(budget=3)}.get(name, dict(scale=0.1))


def run_with_fakes(pa, monkeypatch, name, given):
    log = []
    current = FakeStream(log, "current")
    stream = {"other": FakeStream(log, "other"), "current": current, "none": None}[given]
    plan, n, made = CALLS[name]
    monkeypatch.setattr(pa, plan, fake_plan(log))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    getattr(pa, name)(*[None] * n, **keywords(name), stream=stream)
    return log, made


@pytest.mark.parametrize("name", CALLS)
def test_another_stream_waits_for_the_one_that_allocates(pa, monkeypatch, name):
    log, made = run_with_fakes(pa, monkeypatch, name, "other")
    assert log[0] == "made" and "run on other" in log
    assert log.index("other waits for current") < log.index("run on other")
    for t in made:
        assert f"{t} kept for other" in log, t


@pytest.mark.parametrize("given", ["current", "none"])
@pytest.mark.parametrize("name", CALLS)
def test_the_current_stream_needs_no_wait(pa, monkeypatch, name, given):
    log, _ = run_with_fakes(pa, monkeypatch, name, given)
    assert log[0] == "made" and not any("waits" in x for x in log)


def test_decode_positions_waits(pa, monkeypatch):
    log = []
    current, other = FakeStream(log, "current"), FakeStream(log, "other")
    monkeypatch.setattr(pa, "Plan", fake_plan(log))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(pa, "LIB", types.SimpleNamespace(pa_decode_positions=lambda *a: log.append("run") or 0))
    slots = types.SimpleNamespace(dtype=torch.int32, shape=(2, 1), is_cuda=True, is_contiguous=lambda: True, data_ptr=lambda: 64)
    q = types.SimpleNamespace(shape=(2, 4, 1, 64))
    pa.decode_positions(q, *[None] * 6, slots, scale=0.1, stream=other)
    assert log.index("made") < log.index("other waits for current") < log.index("run")
    assert "out kept for other" in log and "workspace kept for other" in log


def test_decode_host_waits_for_its_new_workspace(pa, monkeypatch):
    log = []
    current, other = FakeStream(log, "current"), FakeStream(log, "other")
    monkeypatch.setattr(pa, "HostPlan", fake_plan(log))
    monkeypatch.setattr(pa, "_host_plans", {})
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: None)
    cache = types.SimpleNamespace(data_ptr=lambda: 64, shape=(4, 16, 2, 64), device="cuda")
    q = types.SimpleNamespace(shape=(2, 4, 1, 64), dtype=torch.float32)
    table = types.SimpleNamespace(shape=(2, 2))
    pa.decode_host(q, table, None, None, None, k_cache=cache, v_cache=cache, scale=0.1, stream=other)
    assert log == ["made", "other waits for current", "run on other", "synchronize other"]


# ------------------------------------------------------------------ GPU
CYCLES = 40_000_000  # about 20 ms of the current stream


def batch(fmt, lens, H, KV, D, BLOCK, NQ):
    g = torch.Generator().manual_seed(7)
    B, per = len(lens), [-(-(n + NQ) // BLOCK) for n in lens]
    table = torch.zeros(B, max(per), dtype=torch.int32)
    perm = torch.randperm(sum(per), generator=g).to(torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = perm[at:at + n]
        at += n
    r = lambda *s: torch.randn(*s, generator=g).to(fmt)  # noqa: E731
    x = (r(B, H, NQ, D), r(sum(per), BLOCK, KV, D), r(sum(per), BLOCK, KV, D), table, torch.tensor(lens, dtype=torch.int32),
         r(B, KV, NQ, D), r(B, KV, NQ, D))
    return [t.cuda() for t in x]


def used_memory(*sizes):
    """Leaves freed blocks of these many bytes, full of ones, to the allocator."""
    for n in sizes:
        torch.full((max(int(n), 1),), 0x01, dtype=torch.uint8, device="cuda")


def while_the_current_stream_is_busy(call, *sizes):
    """call(stream) on a side stream behind a busy current stream; its results, copied on that stream."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    used_memory(*sizes)
    torch.cuda._sleep(CYCLES)
    got = call(side)
    used_memory(*sizes)  # memory that the call has given back must not be written yet
    with torch.cuda.stream(side):
        got = [t.clone() for t in (got if isinstance(got, tuple) else (got,)) if t is not None]
    side.synchronize()
    torch.cuda.synchronize()
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["decode", "decode_scored", "weights", "positions", "prefill"])
def test_decodes_on_another_stream(pa, kind):
    # one long sequence among short ones: segments that are split and merged by counters in the workspace
    NQ = 1 if kind != "prefill" else 5
    x = batch(torch.float16, [9000, 40, 700], 8, 2, 128, 16, NQ)
    slots, slopes = torch.full((3, 1), -1, dtype=torch.int32, device="cuda"), torch.full((8,), 0.1, device="cuda")
    width = x[3].shape[1] * 16
    kw = dict(scale=1 / math.sqrt(128))
    call = {
        "decode": lambda s: pa.decode(*x, **kw, causal=True, stream=s),
        "decode_scored": lambda s: pa.decode_scored(*x, **kw, causal=True, softcap=20.0, stream=s),
        "weights": lambda s: pa.decode_scored(*x, **kw, causal=True, slopes=slopes, stream=s,
                                              key_weights_out=torch.zeros(3, width, device="cuda")),
        "positions": lambda s: pa.decode_positions(*x, slots, **kw, causal=True, stream=s),
        "prefill": lambda s: pa.prefill(*x, **kw, stream=s),
    }[kind]
    want = call(None)
    want = want if isinstance(want, tuple) else (want,)
    torch.cuda.synchronize()
    need = pa.workspace_bytes(3, 8, 2, 128, NQ)
    for _ in range(3):
        got = while_the_current_stream_is_busy(call, need, x[0].numel() * 2, 4 * 3 * width)
        for a, b in zip(want, got):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_gradients_on_another_stream(pa):
    g = torch.Generator().manual_seed(3)
    q, k, v, y, d = (torch.randn(1, h, 300, 64, generator=g).cuda() for h in (4, 2, 2, 4, 4))
    mask = torch.rand(1, 1, 300, 300, generator=g) < 0.8
    mask[..., 0] = True  # every row sees a key, as y does
    mask = mask.cuda()
    far = (torch.arange(300)[:, None] - torch.arange(300)).abs().cuda()
    for window, call in ((300, lambda s: pa.attention_vjp(q, k, v, y, d, mask, scale=0.1, stream=s)),
                         (200, lambda s: pa.attention_vjp_scored(q, k, v, y, d, mask, scale=0.1, window=200, stream=s))):
        want = call(None)
        torch.cuda.synchronize()
        got = while_the_current_stream_is_busy(call, mask.numel(), q.numel() * 4, k.numel() * 4)
        # dk and dv have one order of sums
        assert torch.equal(want[1], got[1]) and torch.equal(want[2], got[2])
        # dq is the sum of 10 tiles' parts in any order: each order is off by at most 9 roundings of
        # the sum of the parts' magnitudes, which is at most |ds| |k|
        Q, K, V, Y, G = (t.double().repeat_interleave(4 // t.shape[1], 1) for t in (q, k, v, y, d))
        p = torch.softmax((0.1 * Q @ K.mT).masked_fill(~mask | (far >= window), -math.inf), -1).nan_to_num(0.0)
        ds = 0.1 * p * (G @ V.mT - (Y * G).sum(-1, keepdim=True))
        assert torch.all((want[0] - got[0]).abs() <= 20 * 2.0 ** -24 * (ds.abs() @ K.abs()) + 2.0 ** -120)


@pytest.mark.gpu
def test_rotary_and_eviction_on_another_stream(pa):
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(2, h, 3, 64, generator=g).cuda() for h in (4, 2, 2))
    pos = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    slots = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    kc, vc = torch.zeros(4, 16, 2, 64, device="cuda"), torch.zeros(4, 16, 2, 64, device="cuda")
    table = pa.rotary_table(64)
    blocks = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    fresh = torch.tensor([[4], [5]], dtype=torch.int32, device="cuda")
    big = [torch.randn(6, 16, 2, 64, generator=g).cuda() for _ in range(2)]
    lens = torch.tensor([30, 20], dtype=torch.int32, device="cuda")
    weights = torch.rand(2, 32, generator=g).cuda()
    for call in (lambda s: pa.rotary(q, k, pos, table, stream=s),
                 lambda s: pa.rotary_append(q, k, v, pos, slots, kc, vc, table, stream=s),
                 lambda s: pa.cache_evict(*big, blocks, lens, weights, budget=12, keep_last=2, dst_table=fresh, stream=s)):
        want = call(None)
        torch.cuda.synchronize()
        for a, b in zip(want, while_the_current_stream_is_busy(call, q.numel() * 4, k.numel() * 4, 256)):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_stream_object_of_another_library(pa):
    # anything with a cuda_stream handle
    x = batch(torch.float16, [700, 40], 4, 2, 64, 16, 1)
    want = pa.decode(*x, scale=0.1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = pa.decode(*x, scale=0.1, stream=types.SimpleNamespace(cuda_stream=side.cuda_stream))
    side.synchronize()
    assert torch.equal(want, got)
    got = pa.decode_scored(*x, scale=0.1, stream=types.SimpleNamespace(cuda_stream=side.cuda_stream))
    side.synchronize()
    assert torch.equal(want, got)
