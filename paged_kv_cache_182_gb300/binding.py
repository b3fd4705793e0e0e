"""ctypes binding of ``libpadecode.so`` (C ABI in ``include/pa_decode.h``).

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  If the library has not been built, importing this
module raises -- there is no Python or CPU fallback.

Tensor layouts (row-major, contiguous):
  q, out           [B, H, NQ, D]            float32 / float16 / bfloat16
  k_cache, v_cache [num_blocks, BLOCK, KV, D]
  block_table      [B, max_blocks]          int32
  seq_lens         [B]                      int32 (cached tokens per sequence)
  k_new, v_new     [B, KV, NQ, D]

Entry points: ``decode`` / ``Plan`` (device tensors), ``decode_host`` /
``HostPlan`` (host tensors, device-resident caches), ``cache_append`` (new
rows into their cache slots), ``decode_positions`` (a decode step with slot
patching), ``prefill`` / ``PrefillPlan`` (causal prefill of any number of
new rows up to PA_MAX_PREFILL) and ``attention_vjp`` / ``VjpPlan`` (dense
attention backward, ``include/pa_attention_vjp.h``: q, y, g [B, HQ, SQ, D],
k, v [B, HK, SK, D]).

Around them: ``rotary`` / ``RotaryPlan`` and ``rotary_append`` /
``RotaryAppendPlan`` (rotary positions, their gradient, and with the store of
the new rows in the cache, ``include/pa_rotary.h``), ``decode_scored`` /
``ScoredPlan`` and ``attention_vjp_scored`` / ``ScoredVjpPlan`` (decode and
backward with scores that are capped, biased by distance or limited to a
window beside a prefix; the decode also accumulates the weight of every key,
``include/pa_scored.h``) and ``cache_evict`` / ``EvictPlan`` (sequences
shortened to their most attended keys, ``include/pa_evict.h``).
"""
from __future__ import annotations

import ctypes
import math
from pathlib import Path

import torch

from . import _build

PA_F32, PA_F16, PA_BF16 = 0, 1, 2
PA_STATUS_BAD_BLOCK, PA_STATUS_BAD_LENGTH, PA_STATUS_TIMEOUT, PA_STATUS_BAD_SLOT = 1, 2, 4, 8
PA_MAX_NQ = 16
PA_MAX_PREFILL = 65536
_DT = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16}

LIBRARY = _build.LIBRARY


class PaOpts(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int),
        ("max_blocks", ctypes.c_int),
        ("num_blocks", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int),
        ("partitions", ctypes.c_int),
        ("checked", ctypes.c_int),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("status", ctypes.c_void_p),
        ("trace_begin", ctypes.c_void_p),
        ("trace_split", ctypes.c_void_p),
        ("merge_kernel", ctypes.c_int),
        ("wait_limit_ns", ctypes.c_ulonglong),
        ("debug_withhold_stage", ctypes.c_int),
        ("inputs_unchanged", ctypes.c_int),
        ("kernel", ctypes.c_int),
    ]


class VjpOpts(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int),
        ("out_dtype", ctypes.c_int),
        ("causal", ctypes.c_int),
        ("mask_kind", ctypes.c_int),
        ("mask_dims", ctypes.c_int * 4),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("status", ctypes.c_void_p),
        ("kernel", ctypes.c_int),
        ("wait_limit_ns", ctypes.c_ulonglong),
    ]


class RotaryOpts(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int),
        ("interleaved", ctypes.c_int),
        ("inverse", ctypes.c_int),
        ("factor", ctypes.c_float),
        ("q_strides", ctypes.c_longlong * 3),
        ("k_strides", ctypes.c_longlong * 3),
        ("v_strides", ctypes.c_longlong * 3),
        ("slot_mapping", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("k_cache", ctypes.c_void_p),
        ("v_cache", ctypes.c_void_p),
        ("BLOCK", ctypes.c_int),
        ("num_blocks", ctypes.c_int),
        ("status", ctypes.c_void_p),
    ]


class EvictOpts(ctypes.Structure):
    _fields_ = [
        ("max_blocks", ctypes.c_int),
        ("num_blocks", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("budget", ctypes.c_int),
        ("keep_first", ctypes.c_int),
        ("keep_last", ctypes.c_int),
        ("dst_table", ctypes.c_void_p),
        ("dst_max_blocks", ctypes.c_int),
        ("status", ctypes.c_void_p),
    ]


class Score(ctypes.Structure):
    _fields_ = [
        ("softcap", ctypes.c_float),
        ("window", ctypes.c_int),
        ("slopes", ctypes.c_void_p),
        ("prefix", ctypes.c_void_p),
    ]


class KeyWeights(ctypes.Structure):
    _fields_ = [
        ("in_", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("decay", ctypes.c_float),
        ("scratch", ctypes.c_void_p),
        ("scratch_bytes", ctypes.c_size_t),
    ]


class SplitPlan(ctypes.Structure):
    _fields_ = [(name, ctypes.c_int) for name in (
        "grid", "active", "segments", "pieces", "split_segments", "records", "max_pieces")]


def load(path: Path = LIBRARY) -> ctypes.CDLL:
    """Load the C-ABI library and declare its signatures."""
    if not Path(path).exists():
        raise RuntimeError(
            f"{path} is missing: build it with paged_kv_cache_182_gb300._build.build() "
            "(there is no fallback path)")
    lib = ctypes.CDLL(str(path))
    P, I = ctypes.c_void_p, ctypes.c_int
    lib.pa_decode.restype = I
    lib.pa_decode.argtypes = [P, P, P, P, P, P, P, P, ctypes.c_float, I, I, I, I, I, I,
                              ctypes.POINTER(PaOpts), P]
    lib.pa_decode_positions.restype = I
    lib.pa_decode_positions.argtypes = [P, P, P, P, P, P, P, P, P, ctypes.c_float, I, I, I, I,
                                        I, I, ctypes.POINTER(PaOpts), P]
    lib.pa_prefill.restype = I
    lib.pa_prefill.argtypes = [P, P, P, P, P, P, P, P, ctypes.c_float, I, I, I, I, I,
                               ctypes.POINTER(PaOpts), P]
    lib.pa_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.pa_prefill_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I]
    lib.pa_prefill_workspace_zero_bytes.restype = ctypes.c_size_t
    lib.pa_prefill_workspace_zero_bytes.argtypes = [I, I, I, I, I, I, I, I]
    lib.pa_decode_static_workspace.restype = I
    lib.pa_decode_static_workspace.argtypes = lib.pa_decode.argtypes
    lib.pa_workspace_bytes.restype = ctypes.c_size_t
    lib.pa_workspace_bytes.argtypes = [I, I, I, I, I, I]
    lib.pa_workspace_zero_bytes.restype = ctypes.c_size_t
    lib.pa_workspace_zero_bytes.argtypes = [I, I, I, I, I, I]
    lib.pa_decode_host.restype = I
    lib.pa_decode_host.argtypes = lib.pa_decode.argtypes
    lib.pa_host_workspace_bytes.restype = ctypes.c_size_t
    lib.pa_host_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I, I]
    lib.pa_strerror.restype = ctypes.c_char_p
    lib.pa_strerror.argtypes = [I]
    lib.pa_version.restype = I
    lib.pa_kernel_launches.restype = ctypes.c_uint64
    lib.pa_host_register.restype = I
    lib.pa_host_register.argtypes = [P, ctypes.c_size_t]
    lib.pa_host_unregister.restype = I
    lib.pa_host_unregister.argtypes = [P]
    lib.pa_choose_partitions.restype = I
    lib.pa_choose_partitions.argtypes = [P, I, I, I, I, I, I, I, I, I, ctypes.POINTER(SplitPlan)]
    lib.pa_attention_vjp.restype = I
    lib.pa_attention_vjp.argtypes = [P, P, P, P, P, P, P, P, P, ctypes.c_float, I, I, I, I, I, I,
                                     ctypes.POINTER(VjpOpts), P]
    lib.pa_attention_vjp_workspace_bytes.restype = ctypes.c_size_t
    lib.pa_attention_vjp_workspace_bytes.argtypes = [I, I, I, I, I, I]
    lib.pa_decode_scored.restype = I
    lib.pa_decode_scored.argtypes = [P, P, P, P, P, P, P, P, ctypes.c_float, I, I, I, I, I, I,
                                     ctypes.POINTER(Score), ctypes.POINTER(KeyWeights),
                                     ctypes.POINTER(PaOpts), P]
    lib.pa_scored_scratch_bytes.restype = ctypes.c_size_t
    lib.pa_scored_scratch_bytes.argtypes = [I, I, I, I, I, I]
    lib.pa_attention_vjp_scored.restype = I
    lib.pa_attention_vjp_scored.argtypes = [P, P, P, P, P, P, P, P, P, ctypes.c_float, I, I, I, I, I, I,
                                            ctypes.POINTER(Score), ctypes.POINTER(VjpOpts), P]
    lib.pa_attention_vjp_scored_workspace_bytes.restype = ctypes.c_size_t
    lib.pa_attention_vjp_scored_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I]
    lib.pa_rotary.restype = I
    lib.pa_rotary.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, ctypes.POINTER(RotaryOpts), P]
    lib.pa_cache_evict.restype = I
    lib.pa_cache_evict.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, ctypes.POINTER(EvictOpts), P]
    lib.pa_cache_append.restype = I
    lib.pa_cache_append.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, P, P]
    return lib


LIB = load()


class PagedAttentionError(RuntimeError):
    def __init__(self, code: int):
        self.code = code
        super().__init__(f"pa_decode returned {code}: {strerror(code)}")


def strerror(code: int) -> str:
    return LIB.pa_strerror(int(code)).decode()


def kernel_launches() -> int:
    return int(LIB.pa_kernel_launches())


def choose_partitions(seq_lens, max_len: int, H: int, KV: int, D: int, BLOCK: int, NQ: int,
                      dtype=torch.float16, sms: int = 0, batch: int | None = None) -> SplitPlan:
    """The automatic split pa_decode makes of a batch with these host lengths
    (pa_choose_partitions); ``seq_lens=None`` means every sequence holds
    ``max_len`` tokens (then ``batch`` gives their number)."""
    if seq_lens is None:
        arr, B = None, int(batch)
    else:
        lens = torch.as_tensor(seq_lens, dtype=torch.int32).contiguous().cpu()
        arr, B = ctypes.c_void_p(lens.data_ptr()), int(lens.numel())
    plan = SplitPlan()
    rc = LIB.pa_choose_partitions(arr, int(max_len), B, H, KV, D, BLOCK, NQ, _DT[dtype], int(sms),
                                  ctypes.byref(plan))
    if rc < 0:
        raise PagedAttentionError(rc)
    return plan


def workspace_bytes(B: int, H: int, KV: int, D: int, NQ: int, partitions: int = 0) -> int:
    return int(LIB.pa_workspace_bytes(B, H, KV, D, NQ, partitions))


def workspace_zero_bytes(B: int, H: int, KV: int, D: int, NQ: int, partitions: int = 0) -> int:
    """Leading workspace bytes that must be zero before first use (in-kernel merge)."""
    return int(LIB.pa_workspace_zero_bytes(B, H, KV, D, NQ, partitions))


def new_workspace(B, H, KV, D, NQ, partitions=0, device="cuda"):
    """A zero-filled workspace of the size pa_decode needs (None when none is needed)."""
    need = workspace_bytes(B, H, KV, D, NQ, partitions)
    return torch.zeros(need, dtype=torch.uint8, device=device) if need > 0 else None


def _ptr(t):
    return None if t is None or t.data_ptr() == 0 else ctypes.c_void_p(t.data_ptr())


def _writable(device, **tensors):
    """Refuses what kernels on ``device`` may not write: memory of another device,
    or host memory that is not pinned."""
    for name, t in tensors.items():
        if t is not None and not (t.device == device if t.is_cuda else t.is_pinned()):
            raise ValueError(f"{name} must be on the inputs' device")


def _status_ptr(status, device):
    """Address of the int32 status word of a call, or None."""
    if status is None:
        return None
    _writable(device, status=status)
    if status.dtype != torch.int32 or status.numel() < 1:
        raise ValueError("status must be an int32 scalar")
    return status.data_ptr()


def _int32(**values):
    """Refuses sizes that the C ABI's int would take for others."""
    for name, v in values.items():
        if not -(2 ** 31) <= v < 2 ** 31:
            raise ValueError(f"{name} is out of range")


def _stream_handle(stream):
    # the raw handle of torch's current stream: building a Stream object costs
    # as much host time as the launch
    if stream is None:
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(torch.cuda.current_device()))
    return ctypes.c_void_p(stream.cuda_stream)


def _ready(args):
    """Arguments that ctypes passes on as they are (plain ints are converted anew by every call)."""
    return tuple(ctypes.c_int(a) if type(a) is int else a for a in args)


def _call(fn, args, device, stream):
    """fn(*args, stream) with the plan's device current; raises on an error code."""
    index = torch.cuda.current_device()
    if index == device.index:
        rc = fn(*args, ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(index) if stream is None
                                       else stream.cuda_stream))
    else:
        with torch.cuda.device(device):
            rc = fn(*args, _stream_handle(stream))
    if rc != 0:
        raise PagedAttentionError(rc)


def _order(stream, device, *made):
    """Orders a call on ``stream`` behind torch's current stream, where the call's
    own tensors ``made`` are allocated, zero-filled or converted (their memory may
    still be in use there); they stay allocated until ``stream`` has passed what
    it holds by the time they are freed."""
    if stream is None:
        return
    if not hasattr(stream, "wait_stream"):  # another library's stream object: its handle is enough
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    current = torch.cuda.current_stream(device)
    if stream == current:
        return
    stream.wait_stream(current)
    for t in made:
        if t is not None:
            t.record_stream(stream)


def _run_once(plan, stream, *made):
    """``plan.run(stream)`` of a plan that was made for this call and is dropped
    right after; ``made``: the tensors that it allocated."""
    _order(stream, plan.device, *made)
    return plan.run(stream)


class Plan:
    """One prepared decode call on fixed device tensors.

    Validates shapes once and packs the ctypes arguments, so that repeated
    calls (a decode loop, CUDA-graph capture, the bench) cost one foreign
    call.  The workspace is allocated once, here, with torch, and zero-filled
    on torch's current stream: a first ``run`` on another stream has to be
    ordered behind that (``stream.wait_stream``).  The one-call functions do it
    themselves.  The same holds for the other plans of this module.
    """

    def __init__(self, q, k_cache, v_cache, block_table, seq_lens, k_new, v_new, *,
                 scale: float, causal: bool = False, partitions: int = 0, out=None,
                 out_dtype=None, workspace=None, status=None, checked: bool = False,
                 trace=None, merge_kernel: bool = False, inputs_unchanged: bool = False,
                 kernel: int = 0):
        B, H, NQ, D = q.shape
        NB, BLOCK, KV, D2 = k_cache.shape
        if (D2 != D or tuple(v_cache.shape) != tuple(k_cache.shape)
                or tuple(k_new.shape) != (B, KV, NQ, D) or tuple(v_new.shape) != (B, KV, NQ, D)):
            raise ValueError("inconsistent q / cache / new-row shapes")
        if block_table.dim() != 2 or block_table.shape[0] != B or tuple(seq_lens.shape) != (B,):
            raise ValueError("block_table must be [B, max_blocks] and seq_lens [B]")
        if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
            raise TypeError("block_table and seq_lens must be int32")
        dt = q.dtype
        for t in (k_cache, v_cache, k_new, v_new):
            if t.dtype != dt:
                raise TypeError("q, caches and new rows must share one dtype")
        if dt not in _DT:
            raise TypeError(f"unsupported dtype {dt}")
        tensors = (q, k_cache, v_cache, block_table, seq_lens, k_new, v_new)
        for t in tensors:
            if not t.is_cuda:
                raise ValueError("all tensors must be CUDA tensors")
            if not t.is_contiguous():
                raise ValueError("all tensors must be contiguous")
        odt = dt if out_dtype is None else out_dtype
        if out is None:
            out = torch.empty((B, H, NQ, D), dtype=odt, device=q.device)
        elif tuple(out.shape) != (B, H, NQ, D) or not out.is_contiguous() or out.dtype != odt:
            raise ValueError("out must be a contiguous [B, H, NQ, D] tensor of the output dtype")
        _writable(q.device, out=out, workspace=workspace)
        if workspace is None:
            workspace = new_workspace(B, H, KV, D, NQ, partitions, q.device)
        self.tensors = tensors
        self.out = out
        self.workspace = workspace
        self.status = status
        self.trace = trace
        self.device = q.device
        self.shape = dict(B=B, H=H, KV=KV, D=D, BLOCK=BLOCK, NQ=NQ, num_blocks=NB,
                          max_blocks=int(block_table.shape[1]))
        self.opts = PaOpts(
            batch=B, max_blocks=int(block_table.shape[1]), num_blocks=NB, dtype=_DT[dt],
            out_dtype=_DT[odt], partitions=int(partitions), checked=int(bool(checked)),
            workspace=None if workspace is None else workspace.data_ptr(),
            workspace_bytes=0 if workspace is None else workspace.numel(),
            status=_status_ptr(status, q.device),
            trace_begin=None if trace is None else trace[0].cuda_event,
            trace_split=None if trace is None else trace[1].cuda_event,
            merge_kernel=int(bool(merge_kernel)), inputs_unchanged=int(bool(inputs_unchanged)),
            kernel=int(kernel))
        self._args = [_ptr(t) for t in tensors] + [_ptr(out), ctypes.c_float(scale), H, KV, D,
                                                   BLOCK, NQ, int(bool(causal)),
                                                   ctypes.byref(self.opts)]

    def set_trace(self, begin=None, split=None):
        """Events recorded around the partition kernel by the next run()."""
        self.opts.trace_begin = None if begin is None else begin.cuda_event
        self.opts.trace_split = None if split is None else split.cuda_event

    def bind_stream(self, stream=None):
        """Fix the stream of later run_bound() calls (default: torch's current)."""
        self._bound = self._args + [_stream_handle(stream)]

    def run_bound(self):
        """Launch on the stream fixed by bind_stream(): one foreign call, no lookups."""
        rc = LIB.pa_decode(*self._bound)
        if rc != 0:
            raise PagedAttentionError(rc)
        return self.out

    def run(self, stream=None):
        """Launch on ``stream`` (default: torch's current stream); returns ``out``."""
        if torch.cuda.current_device() == self.device.index:
            rc = LIB.pa_decode(*self._args, _stream_handle(stream))
        else:
            with torch.cuda.device(self.device):
                rc = LIB.pa_decode(*self._args, _stream_handle(stream))
        if rc != 0:
            raise PagedAttentionError(rc)
        return self.out


def decode(q, k_cache, v_cache, block_table, seq_lens, k_new, v_new, *, scale: float,
           causal: bool = False, partitions: int = 0, out=None, out_dtype=None, workspace=None,
           status=None, checked: bool = False, stream=None, merge_kernel: bool = False,
           kernel: int = 0):
    """Decode attention on device tensors (see the module docstring); returns ``out``.

    A caller-provided ``workspace`` must be zero-filled before its first use
    (see pa_opts.workspace); ``new_workspace`` makes one.  ``kernel`` is
    pa_opts.kernel (0 automatic, 1 the mma.sync kernels only)."""
    plan = Plan(q, k_cache, v_cache, block_table, seq_lens, k_new, v_new, scale=scale,
                causal=causal, partitions=partitions, out=out, out_dtype=out_dtype,
                workspace=workspace, status=status, checked=checked, merge_kernel=merge_kernel,
                kernel=kernel)
    return _run_once(plan, stream, plan.out, plan.workspace)


def decode_positions(q, k_cache, v_cache, block_table, seq_lens, k_new, v_new, positions, *,
                     scale: float, causal: bool = False, partitions: int = 0, out=None,
                     out_dtype=None, workspace=None, status=None, checked: bool = False,
                     stream=None, merge_kernel: bool = False):
    """A decode step with slot patching (pa_decode_positions): new row j of
    sequence b is bound for cache slot positions[b, j] (physical block * BLOCK
    + offset, or -1).  Stores the new rows at their slots in ``k_cache`` /
    ``v_cache`` and attends over the updated cache, so that a cached key whose
    slot a new row of its sequence is bound for reads that row (the last such
    row wins).  ``positions``: int32 [B, NQ] on the device.  Other arguments
    as ``decode``; returns ``out``."""
    plan = Plan(q, k_cache, v_cache, block_table, seq_lens, k_new, v_new, scale=scale,
                causal=causal, partitions=partitions, out=out, out_dtype=out_dtype,
                workspace=workspace, status=status, checked=checked, merge_kernel=merge_kernel)
    B, _, NQ, _ = q.shape
    if positions.dtype != torch.int32 or tuple(positions.shape) != (B, NQ):
        raise ValueError("positions must be an int32 [B, NQ] tensor")
    if not (positions.is_cuda and positions.is_contiguous()):
        raise ValueError("positions must be a contiguous CUDA tensor")
    args = plan._args[:7] + [_ptr(positions)] + plan._args[7:]
    _order(stream, plan.device, plan.out, plan.workspace)
    with torch.cuda.device(plan.device):
        rc = LIB.pa_decode_positions(*args, _stream_handle(stream))
    if rc != 0:
        raise PagedAttentionError(rc)
    return plan.out


class PrefillPlan:
    """One prepared prefill call (pa_prefill) on fixed device tensors: NQ new
    rows per sequence after ``seq_lens`` cached tokens, causal, any NQ up to
    PA_MAX_PREFILL.  ``run`` stores the new rows in the caches at the slots
    the block table gives tokens seq_lens[b] + j and writes the attention
    output into ``out``; the workspace is allocated (zeroed) here."""

    def __init__(self, q, k_cache, v_cache, block_table, seq_lens, k_new, v_new, *,
                 scale: float, partitions: int = 0, out=None, out_dtype=None, status=None,
                 checked: bool = False):
        B, H, NQ, D = q.shape
        NB, BLOCK, KV, D2 = k_cache.shape
        if (D2 != D or tuple(v_cache.shape) != tuple(k_cache.shape)
                or tuple(k_new.shape) != (B, KV, NQ, D) or tuple(v_new.shape) != (B, KV, NQ, D)):
            raise ValueError("inconsistent q / cache / new-row shapes")
        if block_table.ndim != 2 or block_table.shape[0] != B or tuple(seq_lens.shape) != (B,):
            raise ValueError("block_table must be [B, max_blocks] and seq_lens [B]")
        if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
            raise TypeError("block_table and seq_lens must be int32")
        dt = q.dtype
        if dt not in _DT or any(t.dtype != dt for t in (k_cache, v_cache, k_new, v_new)):
            raise TypeError("q, caches and new rows must share one supported dtype")
        tensors = (q, k_cache, v_cache, block_table, seq_lens, k_new, v_new)
        for t in tensors:
            if not (t.is_cuda and t.is_contiguous()):
                raise ValueError("all tensors must be contiguous CUDA tensors")
        odt = dt if out_dtype is None else out_dtype
        if out is None:
            out = torch.empty((B, H, NQ, D), dtype=odt, device=q.device)
        elif tuple(out.shape) != (B, H, NQ, D) or not out.is_contiguous() or out.dtype != odt:
            raise ValueError("out must be a contiguous [B, H, NQ, D] tensor of the output dtype")
        _writable(q.device, out=out)
        need = int(LIB.pa_prefill_workspace_bytes(B, H, KV, D, NQ, int(partitions), _DT[dt],
                                                  _DT[odt]))
        if need == 0 and B > 0:
            raise ValueError("unsupported sizes")
        self.workspace = torch.zeros(max(need, 1), dtype=torch.uint8, device=q.device)
        self.tensors, self.out, self.status, self.device = tensors, out, status, q.device
        self.opts = PaOpts(
            batch=B, max_blocks=int(block_table.shape[1]), num_blocks=NB, dtype=_DT[dt],
            out_dtype=_DT[odt], partitions=int(partitions), checked=int(bool(checked)),
            workspace=self.workspace.data_ptr(), workspace_bytes=need,
            status=_status_ptr(status, q.device), trace_begin=None,
            trace_split=None, merge_kernel=0)
        self._args = [_ptr(t) for t in tensors] + [_ptr(out), ctypes.c_float(scale), H, KV, D,
                                                   BLOCK, NQ, ctypes.byref(self.opts)]

    def run(self, stream=None):
        with torch.cuda.device(self.device):
            rc = LIB.pa_prefill(*self._args, _stream_handle(stream))
        if rc != 0:
            raise PagedAttentionError(rc)
        return self.out


def prefill(q, k_cache, v_cache, block_table, seq_lens, k_new, v_new, *, scale: float,
            partitions: int = 0, out=None, out_dtype=None, status=None, checked: bool = False,
            stream=None):
    """Causal prefill (pa_prefill): new row j of sequence b is token
    seq_lens[b] + j; output row r attends to keys 0 .. seq_lens[b] + r.  The
    new rows are stored in ``k_cache`` / ``v_cache`` at the slots the block
    table gives their tokens (the table must hold blocks for them).  q
    [B, H, NQ, D], new rows [B, KV, NQ, D]; returns ``out``."""
    plan = PrefillPlan(q, k_cache, v_cache, block_table, seq_lens, k_new, v_new, scale=scale,
                       partitions=partitions, out=out, out_dtype=out_dtype, status=status,
                       checked=checked)
    return _run_once(plan, stream, plan.out, plan.workspace)


class HostPlan:
    """A prepared host-buffer decode (pa_decode_host) for fixed sizes.

    The device-resident KV cache and a device workspace (the split workspace
    plus staging for the step's inputs and output, zero-filled once here) are
    fixed; each ``run`` takes the step's host tensors (pinned for asynchronous
    copies) and enqueues their copies, the decode and the copy of the output
    into ``out`` (host)."""

    def __init__(self, k_cache, v_cache, *, B: int, H: int, NQ: int, max_blocks: int,
                 scale: float, causal: bool = False, partitions: int = 0, out_dtype=None):
        NB, BLOCK, KV, D = k_cache.shape
        dt = k_cache.dtype
        if dt not in _DT or v_cache.dtype != dt or tuple(v_cache.shape) != tuple(k_cache.shape):
            raise TypeError("k_cache and v_cache must share one supported dtype and shape")
        if not (k_cache.is_cuda and k_cache.is_contiguous() and v_cache.is_contiguous()):
            raise ValueError("the caches must be contiguous CUDA tensors")
        odt = dt if out_dtype is None else out_dtype
        need = int(LIB.pa_host_workspace_bytes(B, max_blocks, H, KV, D, NQ, int(partitions),
                                               _DT[dt], _DT[odt]))
        if need == 0 and B > 0:
            raise ValueError("unsupported sizes")
        self.workspace = torch.zeros(max(need, 1), dtype=torch.uint8, device=k_cache.device)
        self.caches = (k_cache, v_cache)
        self.device = k_cache.device
        self.shape = dict(B=B, H=H, KV=KV, D=D, NQ=NQ, max_blocks=max_blocks)
        self.dtype, self.out_dtype = dt, odt
        self.opts = PaOpts(batch=B, max_blocks=max_blocks, num_blocks=NB, dtype=_DT[dt],
                           out_dtype=_DT[odt], partitions=int(partitions), checked=0,
                           workspace=self.workspace.data_ptr(), workspace_bytes=need,
                           status=None, trace_begin=None, trace_split=None, merge_kernel=0)
        self._fixed = (ctypes.c_float(scale), H, KV, D, BLOCK, NQ, int(bool(causal)),
                       ctypes.byref(self.opts))
        self._kc, self._vc = _ptr(k_cache), _ptr(v_cache)

    def register(self, *tensors):
        """Declare pinned host tensors to the library (pa_host_register): their
        device addresses are then not looked up on every step, and an ``out``
        among them is written by the kernels in place.  The plan keeps them
        alive and releases the records in ``close``."""
        if not hasattr(self, "_registered"):
            self._registered = []
        for x in tensors:
            if x.is_cuda or not x.is_contiguous():
                raise ValueError("only contiguous host tensors can be registered")
            rc = LIB.pa_host_register(ctypes.c_void_p(x.data_ptr()), x.numel() * x.element_size())
            if rc != 0:
                raise PagedAttentionError(rc)
            self._registered.append(x)

    def close(self):
        """Release the records of the registered tensors (before freeing them)."""
        for x in getattr(self, "_registered", []):
            LIB.pa_host_unregister(ctypes.c_void_p(x.data_ptr()))
        self._registered = []

    def __del__(self):
        try:
            self.close()
        except Exception:  # interpreter shutdown: the library may be gone
            pass

    def bind(self, q, block_table, seq_lens, k_new, v_new, out, stream=None):
        """Check the step's host tensors once and fix them and the stream for
        ``run_bound`` (a loop that refills the same pinned buffers each step)."""
        self._check(q, block_table, seq_lens, k_new, v_new, out)
        self._bound = (_ptr(q), self._kc, self._vc, _ptr(block_table), _ptr(seq_lens), _ptr(k_new),
                       _ptr(v_new), _ptr(out), *self._fixed, _stream_handle(stream))
        self._bound_out = out

    def run_bound(self):
        """One step on the tensors fixed by ``bind``: one foreign call."""
        rc = LIB.pa_decode_host(*self._bound)
        if rc != 0:
            raise PagedAttentionError(rc)
        return self._bound_out

    def _check(self, q, block_table, seq_lens, k_new, v_new, out):
        s = self.shape
        if (tuple(q.shape) != (s["B"], s["H"], s["NQ"], s["D"]) or
                tuple(block_table.shape) != (s["B"], s["max_blocks"]) or
                tuple(seq_lens.shape) != (s["B"],) or tuple(out.shape) != tuple(q.shape) or
                tuple(k_new.shape) != (s["B"], s["KV"], s["NQ"], s["D"]) or
                tuple(v_new.shape) != tuple(k_new.shape)):
            raise ValueError("step tensors do not match the plan's sizes")
        for x in (q, block_table, seq_lens, k_new, v_new, out):
            if x.is_cuda or not x.is_contiguous():
                raise ValueError("step tensors must be contiguous host tensors")
        if q.dtype != self.dtype or k_new.dtype != self.dtype or v_new.dtype != self.dtype:
            raise TypeError("q and the new rows must have the caches' dtype")
        if out.dtype != self.out_dtype:
            raise TypeError("out must have the plan's output dtype")
        if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
            raise TypeError("block_table and seq_lens must be int32")

    def run(self, q, block_table, seq_lens, k_new, v_new, out, stream=None):
        """Enqueue one step on ``stream`` (default: torch's current stream).  All
        six tensors are host tensors; ``out`` holds the result once the stream
        has been synchronised."""
        self._check(q, block_table, seq_lens, k_new, v_new, out)
        args = (_ptr(q), self._kc, self._vc, _ptr(block_table), _ptr(seq_lens), _ptr(k_new),
                _ptr(v_new), _ptr(out), *self._fixed)
        if torch.cuda.current_device() == self.device.index:
            rc = LIB.pa_decode_host(*args, _stream_handle(stream))
        else:
            with torch.cuda.device(self.device):
                rc = LIB.pa_decode_host(*args, _stream_handle(stream))
        if rc != 0:
            raise PagedAttentionError(rc)
        return out


_host_plans = {}


def decode_host(q, block_table, seq_lens, k_new, v_new, *, k_cache, v_cache, scale: float,
                causal: bool = False, partitions: int = 0, out_dtype=None, stream=None):
    """End-to-end decode step from host tensors through pa_decode_host.

    The KV cache (``k_cache``, ``v_cache``) is device-resident state, as a KV
    cache is; the step's inputs -- q, the block table, the lengths and the
    new rows -- are host tensors (pinned for asynchronous copies).  The copies,
    the kernels and the copy of the output back to pinned host memory are
    enqueued by one library call; the device workspace is kept per size.
    Returns the host output tensor after synchronising the stream.
    """
    B, H, NQ, _ = q.shape
    odt = q.dtype if out_dtype is None else out_dtype
    key = (k_cache.data_ptr(), v_cache.data_ptr(), tuple(k_cache.shape), B, H, NQ,
           int(block_table.shape[1]), float(scale), bool(causal), int(partitions), odt)
    plan = _host_plans.get(key)
    if plan is None:
        plan = HostPlan(k_cache, v_cache, B=B, H=H, NQ=NQ, max_blocks=int(block_table.shape[1]),
                        scale=scale, causal=causal, partitions=partitions, out_dtype=out_dtype)
        _host_plans.clear()  # one plan at a time: it owns a device workspace
        _host_plans[key] = plan
        _order(stream, k_cache.device)  # the workspace is zero-filled on the current stream
    if stream is None:
        stream = torch.cuda.current_stream(k_cache.device)
    out = torch.empty(q.shape, dtype=odt, pin_memory=True)
    plan.run(q, block_table, seq_lens, k_new, v_new, out, stream)
    stream.synchronize()
    return out


def cache_append(k_cache, v_cache, k_new, v_new, slot_mapping, *, status=None, stream=None):
    """Writes the new rows into the paged cache (pa_cache_append): for every
    sequence b, new row j and KV head kh with s = slot_mapping[b, j] >= 0,
    k_cache[s // BLOCK, s % BLOCK, kh] = k_new[b, kh, j] (and the same for V).
    All tensors on one CUDA device: caches [num_blocks, BLOCK, KV, D], new rows
    [B, KV, NQ, D] of the caches' dtype, slot_mapping int32 [B, NQ], status an
    optional int32 device scalar for PA_STATUS_BAD_SLOT.  Enqueued on ``stream``
    (default: torch's current stream)."""
    NB, BLOCK, KV, D = k_cache.shape
    B, kv2, NQ, d2 = k_new.shape
    dt = k_cache.dtype
    if dt not in _DT or v_cache.dtype != dt or k_new.dtype != dt or v_new.dtype != dt:
        raise TypeError("caches and new rows must share one supported dtype")
    if (tuple(v_cache.shape) != tuple(k_cache.shape) or tuple(v_new.shape) != tuple(k_new.shape)
            or kv2 != KV or d2 != D or tuple(slot_mapping.shape) != (B, NQ)):
        raise ValueError("shapes: caches [NB, BLOCK, KV, D], new rows [B, KV, NQ, D], slots [B, NQ]")
    if slot_mapping.dtype != torch.int32:
        raise TypeError("slot_mapping must be int32")
    for x in (k_cache, v_cache, k_new, v_new, slot_mapping):
        if not (x.is_cuda and x.is_contiguous()):
            raise ValueError("all tensors must be contiguous CUDA tensors")
    args = (_ptr(k_cache), _ptr(v_cache), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), B, KV, D,
            NQ, BLOCK, NB, _DT[dt], _status_ptr(status, k_cache.device))
    if torch.cuda.current_device() == k_cache.device.index:
        rc = LIB.pa_cache_append(*args, _stream_handle(stream))
    else:
        with torch.cuda.device(k_cache.device):
            rc = LIB.pa_cache_append(*args, _stream_handle(stream))
    if rc != 0:
        raise PagedAttentionError(rc)


PA_VJP_MASK_NONE, PA_VJP_MASK_BOOL, PA_VJP_MASK_ADD = 0, 1, 2


def vjp_workspace_bytes(B: int, HQ: int, SQ: int, D: int, dtype=torch.bfloat16,
                        out_dtype=None) -> int:
    odt = -1 if out_dtype is None else _DT[out_dtype]
    return int(LIB.pa_attention_vjp_workspace_bytes(B, HQ, SQ, D, _DT[dtype], odt))


class VjpPlan:
    """One prepared attention backward (pa_attention_vjp) on fixed device
    tensors: q, y, g [B, HQ, SQ, D] and k, v [B, HK, SK, D] of one dtype, an
    optional mask (uint8 = boolean, float32 = additive) of dims [MB, MH, MQ, W]
    broadcasting against the scores [B, HQ, SQ, SK].  ``run()`` enqueues the
    kernels and returns (dq, dk, dv); the outputs and the workspace are
    allocated once, here (or given as ``out``)."""

    def __init__(self, q, k, v, y, g, mask=None, *, scale: float, causal: bool = False,
                 out_dtype=None, kernel: int = 0, status=None, wait_limit_ns: int = 0, out=None):
        B, HQ, SQ, D = q.shape
        b2, HK, SK, d2 = k.shape
        dt = q.dtype
        if dt not in _DT or any(t.dtype != dt for t in (k, v, y, g)):
            raise TypeError("q, k, v, y, g must share one supported dtype")
        if (b2 != B or d2 != D or tuple(v.shape) != tuple(k.shape) or tuple(y.shape) != tuple(q.shape)
                or tuple(g.shape) != tuple(q.shape)):
            raise ValueError("shapes: q, y, g [B, HQ, SQ, D]; k, v [B, HK, SK, D]")
        for x in (q, k, v, y, g) + (() if mask is None else (mask,)):
            if not (x.is_cuda and x.is_contiguous()):
                raise ValueError("all tensors must be contiguous CUDA tensors")
        o = VjpOpts()
        o.dtype = _DT[dt]
        odt = dt if out_dtype is None else out_dtype
        o.out_dtype = -1 if out_dtype is None else _DT[out_dtype]
        o.causal = int(bool(causal))
        if mask is None:
            o.mask_kind = PA_VJP_MASK_NONE
        else:
            if mask.dim() != 4:
                raise ValueError("mask must have 4 dims [MB, MH, MQ, W]")
            if mask.dtype == torch.uint8 or mask.dtype == torch.bool:
                mask = mask.to(torch.uint8)
                o.mask_kind = PA_VJP_MASK_BOOL
            elif mask.dtype == torch.float32:
                o.mask_kind = PA_VJP_MASK_ADD
            else:
                raise TypeError("mask must be uint8/bool (boolean) or float32 (additive)")
            for e in range(4):
                o.mask_dims[e] = int(mask.shape[e])
        dev = q.device
        if out is None:
            out = tuple(torch.empty(t.shape, dtype=odt, device=dev) for t in (q, k, k))
        self.dq, self.dk, self.dv = out
        for t, ref in zip(out, (q, k, k)):
            if t.dtype != odt or tuple(t.shape) != tuple(ref.shape) or not t.is_contiguous():
                raise ValueError("out: dq like q, dk and dv like k, of the output dtype")
            _writable(dev, out=t)
        need = self._workspace_bytes(B, HQ, HK, SQ, SK, D, o.dtype, o.out_dtype, dev)
        self.workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        o.workspace = _ptr(self.workspace)
        o.workspace_bytes = int(self.workspace.numel())
        o.status = _status_ptr(status, dev)
        o.kernel = int(kernel)
        o.wait_limit_ns = int(wait_limit_ns)
        self.opts = o
        self.mask = mask  # as the kernels read it: a boolean mask is converted here
        self._keep = (q, k, v, y, g, status)
        self.device = dev
        self._args = (_ptr(q), _ptr(k), _ptr(v), _ptr(y), _ptr(g), _ptr(mask), _ptr(self.dq),
                      _ptr(self.dk), _ptr(self.dv), ctypes.c_float(scale), B, HQ, HK, SQ, SK, D,
                      ctypes.byref(self.opts))

    def _workspace_bytes(self, B, HQ, HK, SQ, SK, D, dtype, out_dtype, device):
        return int(LIB.pa_attention_vjp_workspace_bytes(B, HQ, SQ, D, dtype, out_dtype))

    def run(self, stream=None):
        if torch.cuda.current_device() == self.device.index:
            rc = LIB.pa_attention_vjp(*self._args, _stream_handle(stream))
        else:
            with torch.cuda.device(self.device):
                rc = LIB.pa_attention_vjp(*self._args, _stream_handle(stream))
        if rc != 0:
            raise PagedAttentionError(rc)
        return self.dq, self.dk, self.dv


def attention_vjp(q, k, v, y, g, mask=None, *, scale: float, causal: bool = False,
                  out_dtype=None, kernel: int = 0, status=None, stream=None, out=None):
    """dq, dk, dv of attention (pa_attention_vjp): see ``VjpPlan``."""
    plan = VjpPlan(q, k, v, y, g, mask, scale=scale, causal=causal, out_dtype=out_dtype,
                   kernel=kernel, status=status, out=out)
    return _run_once(plan, stream, plan.workspace, plan.dq, plan.dk, plan.dv, plan.mask)


# ------------------------------------------------------------------- modified scores
def _score(softcap, slopes, window, prefix, B, H, device):
    """The checked pa_score of a call (the tensors stay with the caller's plan)."""
    _int32(window=int(window))
    if slopes is not None and (tuple(slopes.shape) != (H,) or slopes.dtype != torch.float32):
        raise ValueError("slopes must be a float32 [H] tensor")
    if prefix is not None and (tuple(prefix.shape) != (B,) or prefix.dtype != torch.int32):
        raise ValueError("prefix must be an int32 [B] tensor")
    for t in (slopes, prefix):
        if t is not None and (not t.is_cuda or t.device != device or not t.is_contiguous()):
            raise ValueError("slopes and prefix must be contiguous CUDA tensors on the inputs' device")
    return Score(softcap=float(softcap), window=int(window),
                 slopes=None if slopes is None else slopes.data_ptr(),
                 prefix=None if prefix is None else prefix.data_ptr())


class ScoredPlan(Plan):
    """One prepared decode call with modified scores (pa_decode_scored): as
    ``Plan``, with

      softcap   scores t -> softcap * tanh(t / softcap) (0: none; else
                2^-100 <= |scale| / softcap <= 2^100)
      slopes    float32 [H]: slopes[h] * |row - key| subtracted (None: none)
      window    keys within ``window`` positions of the row only (0: all)
      prefix    int32 [B]: the first prefix[b] keys are visible to every row

    and optionally the weight that every key got, summed over heads and rows:
    ``key_weights`` and ``key_weights_out`` are float32 [B, max_blocks * BLOCK];
    out = decay * key_weights + this step's weights.  Without
    ``key_weights_out``, ``key_weights`` is updated in place; without
    ``key_weights``, the weights start at zero.  ``run()`` returns ``out``, or
    (out, key_weights_out)."""

    def __init__(self, q, k_cache, v_cache, block_table, seq_lens, k_new, v_new, *, scale: float,
                 causal: bool = False, softcap: float = 0.0, slopes=None, window: int = 0,
                 prefix=None, key_weights=None, key_weights_out=None, decay: float = 1.0,
                 partitions: int = 0, out=None, out_dtype=None, workspace=None, status=None,
                 checked: bool = False):
        super().__init__(q, k_cache, v_cache, block_table, seq_lens, k_new, v_new, scale=scale,
                         causal=causal, partitions=partitions, out=out, out_dtype=out_dtype,
                         workspace=workspace, status=status, checked=checked)
        s = self.shape
        self.score = _score(softcap, slopes, window, prefix, s["B"], s["H"], self.device)
        self.key_weights = key_weights if key_weights_out is None else key_weights_out
        self.weights = self.scratch = None
        if self.key_weights is not None:
            for t in (key_weights, self.key_weights):
                if t is not None and (tuple(t.shape) != (s["B"], s["max_blocks"] * s["BLOCK"])
                                      or t.dtype != torch.float32):
                    raise ValueError("key weights must be float32 [B, max_blocks * BLOCK]")
                if t is not None and (not t.is_cuda or t.device != self.device or not t.is_contiguous()):
                    raise ValueError("key weights must be contiguous CUDA tensors on the inputs' device")
            need = int(LIB.pa_scored_scratch_bytes(s["B"], s["max_blocks"], s["BLOCK"], s["H"], s["KV"],
                                                   s["NQ"]))
            self.scratch = torch.empty(max(need, 1), dtype=torch.uint8, device=self.device)
            self.weights = KeyWeights(in_=None if key_weights is None else key_weights.data_ptr(),
                                      out=self.key_weights.data_ptr(), decay=float(decay),
                                      scratch=self.scratch.data_ptr(), scratch_bytes=need)
        self._scored_keep = (slopes, prefix, key_weights)
        self._args = [*_ready(self._args[:-1]), ctypes.byref(self.score),
                      None if self.weights is None else ctypes.byref(self.weights), ctypes.byref(self.opts)]
        self._result = self.out if self.weights is None else (self.out, self.key_weights)

    def run_bound(self):
        rc = LIB.pa_decode_scored(*self._bound)
        if rc != 0:
            raise PagedAttentionError(rc)
        return self._result

    def run(self, stream=None):
        _call(LIB.pa_decode_scored, self._args, self.device, stream)
        return self._result


def decode_scored(q, k_cache, v_cache, block_table, seq_lens, k_new, v_new, *, scale: float,
                  causal: bool = False, softcap: float = 0.0, slopes=None, window: int = 0,
                  prefix=None, key_weights=None, key_weights_out=None, decay: float = 1.0,
                  partitions: int = 0, out=None, out_dtype=None, workspace=None, status=None,
                  checked: bool = False, stream=None):
    """Decode attention with modified scores (pa_decode_scored): see ``ScoredPlan``."""
    plan = ScoredPlan(q, k_cache, v_cache, block_table, seq_lens, k_new, v_new, scale=scale,
                      causal=causal, softcap=softcap, slopes=slopes, window=window, prefix=prefix,
                      key_weights=key_weights, key_weights_out=key_weights_out, decay=decay,
                      partitions=partitions, out=out, out_dtype=out_dtype, workspace=workspace,
                      status=status, checked=checked)
    return _run_once(plan, stream, plan.out, plan.workspace, plan.scratch)


class ScoredVjpPlan(VjpPlan):
    """One prepared attention backward with modified scores
    (pa_attention_vjp_scored): as ``VjpPlan``, with the ``softcap``, ``slopes``
    [HQ], ``window`` and ``prefix`` [B] of ``ScoredPlan``; row i and key j are
    at positions i and j."""

    def __init__(self, q, k, v, y, g, mask=None, *, scale: float, causal: bool = False,
                 softcap: float = 0.0, slopes=None, window: int = 0, prefix=None, out_dtype=None,
                 kernel: int = 0, status=None, wait_limit_ns: int = 0, out=None):
        super().__init__(q, k, v, y, g, mask, scale=scale, causal=causal, out_dtype=out_dtype,
                         kernel=kernel, status=status, wait_limit_ns=wait_limit_ns, out=out)
        self.score = _score(softcap, slopes, window, prefix, int(q.shape[0]), int(q.shape[1]), q.device)
        self._scored_keep = (slopes, prefix)
        self._args = _ready(self._args[:-1]) + (ctypes.byref(self.score), ctypes.byref(self.opts))

    def _workspace_bytes(self, B, HQ, HK, SQ, SK, D, dtype, out_dtype, device):
        with torch.cuda.device(device):
            return int(LIB.pa_attention_vjp_scored_workspace_bytes(B, HQ, HK, SQ, SK, D, dtype, out_dtype))

    def run(self, stream=None):
        _call(LIB.pa_attention_vjp_scored, self._args, self.device, stream)
        return self.dq, self.dk, self.dv


def attention_vjp_scored(q, k, v, y, g, mask=None, *, scale: float, causal: bool = False,
                         softcap: float = 0.0, slopes=None, window: int = 0, prefix=None,
                         out_dtype=None, kernel: int = 0, status=None, stream=None, out=None):
    """dq, dk, dv of attention with modified scores (pa_attention_vjp_scored):
    see ``ScoredVjpPlan``."""
    plan = ScoredVjpPlan(q, k, v, y, g, mask, scale=scale, causal=causal, softcap=softcap,
                         slopes=slopes, window=window, prefix=prefix, out_dtype=out_dtype,
                         kernel=kernel, status=status, out=out)
    return _run_once(plan, stream, plan.workspace, plan.dq, plan.dk, plan.dv, plan.mask)


# ------------------------------------------------------------------- rotary positions
class RotaryTable:
    """Angles per position of a rotary embedding (``rotary_table``): ``turns``
    (int64 [rot / 2] on the device, 2^64 = one turn), the ``factor`` on the
    rotated columns and ``rot``, the columns that turn."""

    def __init__(self, turns, factor: float, rot: int):
        self.turns, self.factor, self.rot = turns, float(factor), int(rot)


def rotary_frequencies(rot: int, *, base: float = 10000.0, scaling=None):
    """(radians per position of the ``rot`` / 2 pairs, factor) in 64 bits.

    Pair i turns by base^(-2 i / rot) per position.  ``scaling`` stretches
    that to contexts longer than the model was trained on:
      None
      ("linear", f)                     every frequency divided by f
      ("ntk", f)                        base times f^(rot / (rot - 2))
      ("bands", f, L, low, high)        pairs with at least ``high`` turns in
                                        the original length L are kept, those
                                        with at most ``low`` divided by f,
                                        those between mixed by their turns
      ("yarn", f, L, fast, slow)        the same by pair index: kept up to the
                                        pair with ``fast`` turns in L, divided
                                        by f from the one with ``slow`` on,
                                        a linear ramp between; factor
                                        0.1 ln f + 1
    """
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    if not base > 1.0:
        raise ValueError("base must be greater than 1")
    kind, args = (None, ()) if scaling is None else (scaling[0], tuple(float(a) for a in scaling[1:]))
    need = {None: 0, "linear": 1, "ntk": 1, "bands": 4, "yarn": 4}
    if kind not in need or len(args) != need[kind] or any(not a > 0.0 for a in args):
        raise ValueError(f"unknown rotary scaling {scaling!r}")
    factor = 1.0
    if kind == "ntk":
        if rot < 4:
            raise ValueError("ntk scaling needs rot >= 4")
        base = base * args[0] ** (rot / (rot - 2))
    inv = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "linear":
        inv = [x / args[0] for x in inv]
    elif kind == "bands":
        f, length, low, high = args
        if not high > low:
            raise ValueError("bands: high must be greater than low")
        for i, x in enumerate(inv):
            keep = min(1.0, max(0.0, (length * x / (2 * math.pi) - low) / (high - low)))
            inv[i] = x * (keep + (1.0 - keep) / f)
    elif kind == "yarn":
        f, length, fast, slow = args
        at = [rot * math.log(length / (2 * math.pi * n)) / (2 * math.log(base)) for n in (fast, slow)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        for i, x in enumerate(inv):
            ramp = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            inv[i] = x * (1.0 - ramp + ramp / f)
        factor = 0.1 * math.log(f) + 1.0
    return inv, factor


# floor(2^256 / (2 pi)): the table entries below need more than 64 bits of 1 / (2 pi)
_INV_2PI = 10 ** 80 * 2 ** 255 // 314159265358979323846264338327950288419716939937510582097494459230781640628620899


def rotary_table(rot: int, *, base: float = 10000.0, scaling=None, device="cuda") -> RotaryTable:
    """The table of a rotary embedding (see ``rotary_frequencies``), made once
    and kept: each pair's angle per position as a 64-bit fraction of a turn."""
    inv, factor = rotary_frequencies(rot, base=base, scaling=scaling)
    turns = []
    for x in inv:
        n, d = x.as_integer_ratio()  # d is a power of two
        turns.append(((n * _INV_2PI // d >> 191) + 1 >> 1) % 2 ** 64)
    signed = [t - 2 ** 64 if t >= 2 ** 63 else t for t in turns]
    return RotaryTable(torch.tensor(signed, dtype=torch.int64, device=device), factor, rot)


def _row_strides(t):
    s = t.stride()
    if t.shape[-1] > 1 and s[3] != 1:
        raise ValueError("the last dimension of q, k and v must be contiguous")
    # a dimension of one element has no stride that matters
    return tuple(0 if n == 1 else int(x) for n, x in zip(t.shape[:3], s[:3]))


class RotaryPlan:
    """One prepared rotary call (pa_rotary) on fixed device tensors: q
    [B, H, N, D] and k [B, KV, N, D] (either may be None) turned by
    ``positions`` (int32 [B, N]).  q and k may be strided views (slices of a
    fused projection) with contiguous columns; the outputs are contiguous.
    ``inverse=True`` turns back: with q and k the gradients arriving at the
    outputs, the result is the gradient of the inputs.  ``run()`` returns
    (q_out, k_out)."""

    def __init__(self, q, k, positions, table: RotaryTable, *, interleaved: bool = False,
                 inverse: bool = False, q_out=None, k_out=None):
        self._prepare(q, k, None, positions, table, interleaved, inverse, q_out, k_out)

    def _prepare(self, q, k, v, positions, table, interleaved, inverse, q_out, k_out, slots=None,
                 caches=None, status=None):
        rows = [t for t in (q, k) if t is not None]
        if not rows or any(t.dim() != 4 for t in rows):
            raise ValueError("shapes: q [B, H, N, D], k [B, KV, N, D]")
        B, _, N, D = rows[0].shape
        H, KV = (0 if t is None else int(t.shape[1]) for t in (q, k))
        dt, dev = rows[0].dtype, rows[0].device
        if dt not in _DT or any(t.dtype != dt for t in rows):
            raise TypeError("q and k must share one supported dtype")
        if tuple(rows[-1].shape) != (B, rows[-1].shape[1], N, D):
            raise ValueError("q and k must agree in batch, rows and head size")
        if tuple(positions.shape) != (B, N) or positions.dtype != torch.int32:
            raise ValueError("positions must be an int32 [B, N] tensor")
        if not positions.is_contiguous():
            raise ValueError("positions must be contiguous")
        if table.rot > D:
            raise ValueError("the table turns more columns than a head has")
        if table.turns.dtype != torch.int64 or table.turns.numel() != table.rot // 2 or not table.turns.is_contiguous():
            raise ValueError("the table must hold rot / 2 int64 angles")
        for t in (*rows, positions, table.turns):
            if not t.is_cuda or t.device != dev:
                raise ValueError("all tensors must be CUDA tensors on one device")
        outs = []
        for t, o in ((q, q_out), (k, k_out)):
            if t is None:
                outs.append(None)
                continue
            if o is None:
                o = torch.empty(t.shape, dtype=dt, device=dev)
            elif tuple(o.shape) != tuple(t.shape) or o.dtype != dt or not o.is_contiguous() or o.device != dev:
                raise ValueError("q_out and k_out must be contiguous tensors like q and k")
            outs.append(o)
        self.q_out, self.k_out = outs
        o = RotaryOpts()
        o.dtype, o.interleaved, o.inverse = _DT[dt], int(bool(interleaved)), int(bool(inverse))
        o.factor = table.factor
        for name, t in (("q_strides", q), ("k_strides", k), ("v_strides", v)):
            if t is not None:
                getattr(o, name)[:] = _row_strides(t)
        if slots is not None:
            o.slot_mapping, o.v = slots.data_ptr(), v.data_ptr()
            o.k_cache, o.v_cache = caches[0].data_ptr(), caches[1].data_ptr()
            o.num_blocks, o.BLOCK = int(caches[0].shape[0]), int(caches[0].shape[1])
            o.status = _status_ptr(status, dev)
        self.opts, self.device = o, dev
        self._keep = (q, k, v, positions, table, slots, caches, status)
        self._args = _ready((_ptr(q), _ptr(k), _ptr(positions), _ptr(table.turns), _ptr(self.q_out),
                             _ptr(self.k_out), B, H, KV, N, D, table.rot, ctypes.byref(self.opts)))

    def run(self, stream=None):
        """Enqueue on ``stream`` (default: torch's current stream); returns (q_out, k_out)."""
        _call(LIB.pa_rotary, self._args, self.device, stream)
        return self.q_out, self.k_out


class RotaryAppendPlan(RotaryPlan):
    """A rotary call that also stores the step's rows in the paged cache: the
    rotated k and the untouched v of row n of sequence b go to slot
    ``slot_mapping[b, n]`` of ``k_cache`` / ``v_cache`` [num_blocks, BLOCK, KV, D]
    (as ``cache_append`` does; -1 stores nothing).  ``run()`` returns the
    rotated (q_out, k_out), ready for ``decode``."""

    def __init__(self, q, k, v, positions, slot_mapping, k_cache, v_cache, table: RotaryTable, *,
                 interleaved: bool = False, q_out=None, k_out=None, status=None):
        if k is None or tuple(v.shape) != tuple(k.shape) or v.dtype != k.dtype:
            raise ValueError("k and v must share one shape and dtype")
        if k_cache.dim() != 4 or tuple(v_cache.shape) != tuple(k_cache.shape) or \
                tuple(k_cache.shape[2:]) != (k.shape[1], k.shape[3]):
            raise ValueError("shapes: caches [num_blocks, BLOCK, KV, D]")
        if k_cache.dtype != k.dtype or v_cache.dtype != k.dtype:
            raise TypeError("the caches must have the dtype of k and v")
        if tuple(slot_mapping.shape) != (k.shape[0], k.shape[2]) or slot_mapping.dtype != torch.int32:
            raise ValueError("slot_mapping must be an int32 [B, N] tensor")
        for t in (v, k_cache, v_cache, slot_mapping):
            if not t.is_cuda or t.device != k.device:
                raise ValueError("all tensors must be CUDA tensors on one device")
        for t in (k_cache, v_cache, slot_mapping):
            if not t.is_contiguous():
                raise ValueError("the caches and slot_mapping must be contiguous")
        self._prepare(q, k, v, positions, table, interleaved, False, q_out, k_out, slot_mapping,
                      (k_cache, v_cache), status)


def rotary(q, k, positions, table: RotaryTable, *, interleaved: bool = False, inverse: bool = False,
           q_out=None, k_out=None, stream=None):
    """q and k turned by their positions (pa_rotary): see ``RotaryPlan``."""
    plan = RotaryPlan(q, k, positions, table, interleaved=interleaved, inverse=inverse, q_out=q_out,
                      k_out=k_out)
    return _run_once(plan, stream, plan.q_out, plan.k_out)


def rotary_append(q, k, v, positions, slot_mapping, k_cache, v_cache, table: RotaryTable, *,
                  interleaved: bool = False, q_out=None, k_out=None, status=None, stream=None):
    """``rotary`` with the store of the new rows in the cache: see ``RotaryAppendPlan``."""
    plan = RotaryAppendPlan(q, k, v, positions, slot_mapping, k_cache, v_cache, table,
                            interleaved=interleaved, q_out=q_out, k_out=k_out, status=status)
    return _run_once(plan, stream, plan.q_out, plan.k_out)


# ------------------------------------------------------------------- cache eviction
class EvictPlan:
    """One prepared eviction (pa_cache_evict) on fixed device tensors: every
    sequence of more than ``budget`` cached tokens keeps its first
    ``keep_first``, its last ``keep_last`` and, of those between, the ones
    with the largest ``key_weights`` (float32 [B, max_blocks * BLOCK], as
    ``ScoredPlan`` accumulates them; equal weights: the lowest index), in
    order.  Their K and V rows move to the sequence's first slots, or with
    ``dst_table`` (int32 [B, dst_max_blocks]) into that table's blocks.

    ``run()`` returns (new_lens [B], kept [B, budget], weights_out like
    ``key_weights``): the shortened lengths, the kept tokens' old indices (-1
    behind them) and their weights (0 behind them).  ``seq_lens`` and
    ``key_weights`` are left as they are: the loop goes on with the returned
    ones.  Rotary positions go on counting the text (cached keys keep theirs);
    the window, slopes and prefix of ``decode_scored`` count places in the
    shortened cache, so ``keep_first`` and ``keep_last`` should cover prefix
    and window where their distances are to stay exact.  Blocks shared between sequences must not be moved in place."""

    def __init__(self, k_cache, v_cache, block_table, seq_lens, key_weights, *, budget: int,
                 keep_first: int = 0, keep_last: int = 0, dst_table=None, new_lens=None, kept=None,
                 weights_out=None, status=None):
        if k_cache.dim() != 4 or tuple(v_cache.shape) != tuple(k_cache.shape):
            raise ValueError("shapes: caches [num_blocks, BLOCK, KV, D]")
        NB, BLOCK, KV, D = k_cache.shape
        if k_cache.dtype not in _DT or v_cache.dtype != k_cache.dtype:
            raise TypeError("k_cache and v_cache must share one supported dtype")
        if block_table.dim() != 2 or tuple(seq_lens.shape) != (block_table.shape[0],):
            raise ValueError("block_table must be [B, max_blocks] and seq_lens [B]")
        B, maxb = (int(x) for x in block_table.shape)
        if dst_table is not None and (dst_table.dim() != 2 or dst_table.shape[0] != B):
            raise ValueError("dst_table must be [B, dst_max_blocks]")
        if any(t.dtype != torch.int32 for t in (block_table, seq_lens, dst_table) if t is not None):
            raise TypeError("block_table, seq_lens and dst_table must be int32")
        if tuple(key_weights.shape) != (B, maxb * BLOCK) or key_weights.dtype != torch.float32:
            raise ValueError("key_weights must be float32 [B, max_blocks * BLOCK]")
        budget = int(budget)
        if budget < 1:
            raise ValueError("budget must be at least 1")
        _int32(budget=budget, keep_first=int(keep_first), keep_last=int(keep_last))
        dev = k_cache.device

        def output(t, shape, dtype, name):
            if t is None:
                return torch.empty(shape, dtype=dtype, device=dev)
            if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
                raise ValueError(f"{name} must be {dtype} {list(shape)}")
            return t

        self.new_lens = output(new_lens, (B,), torch.int32, "new_lens")
        self.kept = output(kept, (B, budget), torch.int32, "kept")
        self.weights_out = output(weights_out, (B, maxb * BLOCK), torch.float32, "weights_out")
        tensors = (k_cache, v_cache, block_table, seq_lens, key_weights, self.new_lens, self.kept,
                   self.weights_out)
        for t in tensors + (() if dst_table is None else (dst_table,)):
            if not t.is_cuda or t.device != dev:
                raise ValueError("all tensors must be CUDA tensors on one device")
            if not t.is_contiguous():
                raise ValueError("all tensors must be contiguous")
        self.opts = EvictOpts(
            max_blocks=maxb, num_blocks=NB, dtype=_DT[k_cache.dtype], budget=budget,
            keep_first=int(keep_first), keep_last=int(keep_last),
            dst_table=None if dst_table is None else dst_table.data_ptr(),
            dst_max_blocks=0 if dst_table is None else int(dst_table.shape[1]),
            status=_status_ptr(status, dev))
        self.device = dev
        self._keep = (tensors, dst_table, status)
        self._args = _ready((*(_ptr(t) for t in tensors), B, KV, D, BLOCK, ctypes.byref(self.opts)))

    def run(self, stream=None):
        """Enqueue on ``stream`` (default: torch's current stream)."""
        _call(LIB.pa_cache_evict, self._args, self.device, stream)
        return self.new_lens, self.kept, self.weights_out


def cache_evict(k_cache, v_cache, block_table, seq_lens, key_weights, *, budget: int,
                keep_first: int = 0, keep_last: int = 0, dst_table=None, status=None, stream=None):
    """Shortens every sequence to its budget (pa_cache_evict): see ``EvictPlan``."""
    plan = EvictPlan(k_cache, v_cache, block_table, seq_lens, key_weights, budget=budget,
                     keep_first=keep_first, keep_last=keep_last, dst_table=dst_table, status=status)
    return _run_once(plan, stream, plan.new_lens, plan.kept, plan.weights_out)
