"""One workspace of pa_q8_decode for calls of unlike sizes in turn: the bytes that
have to be zero are the same for all of them, and stay zero."""
import numpy as np
import pytest
import torch

from test_q8 import Cache, ints, rows_of


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_182_gb300 import _build

    _build.build()
    from paged_kv_cache_182_gb300 import binding

    return binding


def test_the_zero_bytes_are_the_same_for_all_sizes(pa):
    """A call leaves its own zero bytes zero and may write anything behind them."""
    sizes = [(B, H, KV, D, NQ) for B in (1, 64, 4096) for H, KV in ((1, 1), (32, 8), (64, 8)) for D in (64, 128) for NQ in (1, 4, 16)]
    zero = {pa.q8_workspace_zero_bytes(*s) for s in sizes}
    assert len(zero) == 1 and 0 < min(zero) < min(pa.q8_workspace_bytes(*s) for s in sizes)


# one long sequence; long ones behind many short ones; the same with several rows; float32; selected lists
SHAPES = [([20000], 1, 4, 1, 128, "bf16"), ([3] * 61 + [9000, 300, 7000], 8, 1, 1, 64, "f16"), ([5] * 40 + [5000, 2000], 8, 8, 4, 64, "f16"),
          ([1] * 75 + [14000], 2, 2, 1, 128, "f32"), ([0, 16000, 11000], 8, 4, 1, 64, "bf16")]


@pytest.mark.gpu
def test_calls_of_unlike_sizes_in_turn(pa):
    cases, need = [], 0
    for i, (lens, KV, G, NQ, D, fmt) in enumerate(SHAPES):
        c = Cache(50 + i, [16] * len(lens), KV, D, 16)
        c.lens = np.asarray(lens, np.int32)
        c.table = c.rng.integers(0, len(c.ks), (len(lens), -(-max(lens) // 16))).astype(np.int32)  # (blocks may be shared)
        size = (len(lens), KV * G, KV, D, NQ)
        cases.append((c.cuda(), ints(lens), rows_of(c.rng, fmt, len(lens), KV * G, NQ, D).cuda(), size))
        need = max(need, pa.q8_workspace_bytes(*size))
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    zero = pa.q8_workspace_zero_bytes(*cases[0][3])
    plans, want = [], []
    for dev, lens, q, size in cases:
        own = torch.zeros(pa.q8_workspace_bytes(*size), dtype=torch.uint8, device="cuda")
        want.append(pa.decode_q8(q, *dev, lens, scale=0.1, causal=True, workspace=own))
        torch.cuda.synchronize()
        assert bool(own[zero:].any()) and not bool(own[:zero].any())  # pieces were joined
        plans.append(pa.Q8Plan(q, *dev, lens, scale=0.1, causal=True, workspace=ws))
    for order in ((0, 1, 2, 3, 4), (4, 3, 2, 1, 0), (0, 2, 4, 1, 3)):
        for i in order:
            plans[i].out.fill_(float("nan"))
            got = plans[i].run()
            torch.cuda.synchronize()
            assert torch.equal(got, want[i]), i
            assert not bool(ws[:zero].any()), i
