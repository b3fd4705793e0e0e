"""Tensors and sizes that a plan must refuse before anything is launched:
host memory where a kernel would write, status words of another type, angles
that are not the table's, sizes that a C int would take for others."""
import math

import pytest
import torch


@pytest.fixture(scope="module")
def pa():
    from paged_kv_cache_182_gb300 import _build

    _build.build()
    from paged_kv_cache_182_gb300 import binding

    return binding


# ------------------------------------------------------------------ CPU
CUDA = torch.device("cuda", 0)


def test_host_memory_is_not_written(pa):
    with pytest.raises(ValueError, match="out"):
        pa._writable(CUDA, workspace=None, out=torch.zeros(4))
    pa._writable(CUDA, out=None)


def test_status_words(pa):
    assert pa._status_ptr(None, CUDA) is None
    with pytest.raises(ValueError, match="status"):
        pa._status_ptr(torch.zeros(1, dtype=torch.int32), CUDA)


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32 + 5, -(2 ** 31) - 1])
def test_windows_that_no_int_holds(pa, window):
    with pytest.raises(ValueError, match="window"):
        pa._score(0.0, None, window, None, 1, 1, CUDA)


def test_every_other_window_is_passed_on(pa):
    for window in (0, 5, 2 ** 31 - 1, -1):  # (a negative one is the library's to refuse)
        assert pa._score(0.0, None, window, None, 1, 1, CUDA).window == window


# ------------------------------------------------------------------ GPU
def paged(D=64, NQ=1):
    r = lambda *s: torch.randn(*s).half().cuda()  # noqa: E731
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    return [r(2, 4, NQ, D), r(6, 16, 2, D), r(6, 16, 2, D), ints([[0, 1, 2], [3, 4, 5]]), ints([20, 5]), r(2, 2, NQ, D), r(2, 2, NQ, D)]


def calls(pa):
    """Every entry point, as f(status)."""
    x = paged()
    q, k, v, g = (torch.randn(1, h, 20, 64).cuda() for h in (4, 2, 2, 4))
    pos = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    slots = pos - 1
    table = pa.rotary_table(64)
    return {
        "decode": lambda s: pa.decode(*x, scale=0.1, status=s),
        "decode_scored": lambda s: pa.decode_scored(*x, scale=0.1, window=4, status=s),
        "decode_positions": lambda s: pa.decode_positions(*x, slots, scale=0.1, status=s),
        "prefill": lambda s: pa.prefill(*x, scale=0.1, status=s),
        "cache_append": lambda s: pa.cache_append(x[1], x[2], x[5], x[6], slots, status=s),
        "attention_vjp": lambda s: pa.attention_vjp(q, k, v, q, g, scale=0.1, status=s),
        "attention_vjp_scored": lambda s: pa.attention_vjp_scored(q, k, v, q, g, scale=0.1, window=4, status=s),
        "rotary_append": lambda s: pa.rotary_append(x[0], x[5], x[6], pos, slots, x[1], x[2], table, status=s),
        "cache_evict": lambda s: pa.cache_evict(*x[1:5], torch.rand(2, 48, device="cuda"), budget=12, status=s),
    }


@pytest.mark.gpu
def test_status_must_be_a_device_word(pa):
    for name, f in calls(pa).items():
        for bad in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")):
            with pytest.raises(ValueError, match="status"):
                f(bad)
        for good in (torch.zeros((), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32).pin_memory()):
            f(good)
            torch.cuda.synchronize()
            assert int(good) == 0, name


@pytest.mark.gpu
def test_outputs_and_workspaces_on_the_host(pa):
    x = paged()
    host = torch.zeros(2, 4, 1, 64, dtype=torch.float16)
    for f in (lambda **kw: pa.decode(*x, scale=0.1, **kw), lambda **kw: pa.decode_scored(*x, scale=0.1, **kw),
              lambda **kw: pa.prefill(*x, scale=0.1, **kw)):
        with pytest.raises(ValueError, match="out"):
            f(out=host)
    with pytest.raises(ValueError, match="workspace"):
        pa.decode_scored(*x, scale=0.1, workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    q, k, v, g = (torch.randn(1, h, 20, 64).cuda() for h in (4, 2, 2, 4))
    with pytest.raises(ValueError, match="out"):
        pa.attention_vjp_scored(q, k, v, q, g, scale=0.1, out=(torch.zeros(q.shape), torch.zeros(k.shape), torch.zeros(k.shape)))


@pytest.mark.gpu
def test_tables_of_another_length(pa):
    q, pos = torch.randn(1, 2, 3, 64, device="cuda"), torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    turns = pa.rotary_table(64).turns
    for bad in (turns[:31], turns.int(), turns.repeat(2)[::2]):
        with pytest.raises(ValueError, match="angles"):
            pa.rotary(q, None, pos, pa.RotaryTable(bad, 1.0, 64))
    got, _ = pa.rotary(q, None, pos, pa.RotaryTable(turns, 1.0, 64))
    torch.cuda.synchronize()
    assert torch.equal(got, q)  # position 0


@pytest.mark.gpu
def test_sizes_that_no_int_holds(pa):
    x = paged()
    with pytest.raises(ValueError, match="window"):
        pa.decode_scored(*x, scale=1 / math.sqrt(64), window=2 ** 32 + 5)
    for bad in (dict(keep_first=2 ** 32), dict(keep_last=2 ** 32 + 1)):
        with pytest.raises(ValueError, match="keep"):
            pa.cache_evict(*x[1:5], torch.rand(2, 48, device="cuda"), budget=12, **bad)
