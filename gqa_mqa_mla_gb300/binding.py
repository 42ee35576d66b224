"""Python binding of libdecattn (include/decattn.h).

Argument marshalling only: every step of the computation runs in the CUDA
kernels behind the C ABI.  PyTorch supplies device memory and the current
stream.  The GQA decode calls and the serving step's operators are marshalled
natively (csrc/torch_calls.cpp: checks, allocations, stream and call in one
step, for the latency of small calls); the others through ctypes, and the decode
calls too where the native half is missing or was built for another PyTorch.  If
libdecattn is missing the calls raise; there is no fallback implementation.

Every call runs on the current stream of the tensors' device, or on `stream`
where it is given (a torch.cuda.Stream or a handle): inputs must then be ready on
that stream.  What such a call allocates and returns (the GQA decode forms, the
step operators) may be used on the current stream too, once that has waited for
`stream`, and dropped at any time.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import threading
import warnings
from typing import NamedTuple

import torch

from . import build as _build

DECATTN_OK = 0
DECATTN_ERR_INVALID_ARG = -1
DECATTN_ERR_UNSUPPORTED = -2
DECATTN_ERR_WORKSPACE = -3
DECATTN_ERR_CUDA = -4
DECATTN_FP16 = 0
DECATTN_BF16 = 1
FLAG_BAD_BLOCK = 1
FLAG_BAD_SEQ_LEN = 2
FLAG_TIMEOUT = 4
FLAG_NO_ROOM = 8
MAX_SPLITS = 256

MLA_HEADS, MLA_D_C, MLA_D_R = 128, 512, 64

_DT = {torch.float16: DECATTN_FP16, torch.bfloat16: DECATTN_BF16}


class DecAttnError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status_string(status)} ({status})")
        self.status = status


class Launch(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int),
        ("num_blocks", ctypes.c_int),
        ("block_size", ctypes.c_int),
        ("max_blocks_per_seq", ctypes.c_int),
        ("max_seq_len", ctypes.c_int),
        ("num_splits", ctypes.c_int),
        ("dtype", ctypes.c_int),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("err_flag", ctypes.c_void_p),
        ("stream", ctypes.c_void_p),
    ]


class RopeTable(ctypes.Structure):
    """decattn_rope: how a model's heads are rotated (made by rope_table)."""

    _fields_ = [
        ("rot_dim", ctypes.c_int),
        ("n_axes", ctypes.c_int),
        ("interleaved", ctypes.c_int),
        ("axis", ctypes.c_uint8 * 64),
        ("turns", ctypes.c_uint64 * 64),
    ]


class PagedPlan(NamedTuple):
    """What paged_plan writes beside the block table and the free stack."""

    seq_lens: torch.Tensor    # int32 [B]
    q_start: torch.Tensor     # int32 [B + 1]
    slots: torch.Tensor       # int32 [max_tokens]
    positions: torch.Tensor   # int32 [max_tokens]
    free_count: torch.Tensor  # int32 [1]


class Evicted(NamedTuple):
    """What gqa_kv_evict returns beside the caches and weights that it updates."""

    new_lens: torch.Tensor  # int32 [B]: minus the tokens evicted (paged_plan's new_lens)
    kept: torch.Tensor      # int32 [B, h_kv, keep]: old positions; -1: nothing evicted


_lock = threading.Lock()
_lib = None
_calls = None


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Load libdecattn.so (built by gqa_mqa_mla_gb300.build.build())."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = _build.LIB
            if not os.path.exists(path):
                raise RuntimeError(f"{path} is missing: build it with "
                                   "`python -m gqa_mqa_mla_gb300.build` (no fallback exists)")
            L = ctypes.CDLL(path)
            P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
            S, I64 = ctypes.c_size_t, ctypes.c_int64
            LP = ctypes.POINTER(Launch)
            L.gqa_decode.argtypes = [P, P, P, P, P, P, I, I, I, F, LP]
            L.gqa_decode.restype = I
            L.gqa_decode_fp8kv.argtypes = [P, P, P, P, P, P, P, P, I, I, I, F, LP]
            L.gqa_decode_fp8kv.restype = I
            L.gqa_decode_window.argtypes = [P, P, P, P, P, P, I, I, I, F, I, LP]
            L.gqa_decode_window.restype = I
            L.gqa_decode_fp8kv_window.argtypes = [P, P, P, P, P, P, P, P, I, I, I, F, I, LP]
            L.gqa_decode_fp8kv_window.restype = I
            L.gqa_decode_window_plan_splits.argtypes = [I, I, I, I, I, I, I, I, I]
            L.gqa_decode_window_plan_splits.restype = I
            L.gqa_decode_sinks.argtypes = [P, P, P, P, P, P, I, I, I, F, I, I, LP]
            L.gqa_decode_sinks.restype = I
            L.gqa_decode_fp8kv_sinks.argtypes = [P, P, P, P, P, P, P, P, I, I, I, F, I, I, LP]
            L.gqa_decode_fp8kv_sinks.restype = I
            L.gqa_decode_sinks_plan_splits.argtypes = [I, I, I, I, I, I, I, I, I, I]
            L.gqa_decode_sinks_plan_splits.restype = I
            L.paged_plan.argtypes = [P, P, P, P, P, P, P, P, P, P, I, LP]
            L.paged_plan.restype = I
            RP = ctypes.POINTER(RopeTable)
            L.decattn_rope_fill.argtypes = [RP, ctypes.POINTER(ctypes.c_double), I,
                                            ctypes.POINTER(I), I, I]
            L.decattn_rope_fill.restype = I
            L.gqa_rope_append.argtypes = [P, P, P, I64, I64, I64, P, RP, P, P, P, P, I, I, I, I,
                                          LP]
            L.gqa_rope_append.restype = I
            L.gqa_rope_append_fp8kv.argtypes = [P, P, P, I64, I64, I64, P, P, P, RP, P, P, P, P, I,
                                                I, I, I, LP]
            L.gqa_rope_append_fp8kv.restype = I
            L.gqa_prefill.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, F, I, I, LP]
            L.gqa_prefill.restype = I
            L.gqa_prefill_fp8kv.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, F, I, I, LP]
            L.gqa_prefill_fp8kv.restype = I
            L.gqa_prefill_plan_splits.argtypes = [I, I, I, I, I, I, I, I, I, I]
            L.gqa_prefill_plan_splits.restype = I
            L.gqa_prefill_workspace_size.argtypes = [I, I, I, I]
            L.gqa_prefill_workspace_size.restype = S
            L.gqa_decode_blocks.argtypes = [P, P, P, P, P, P, P, I, I, I, F, I, LP]
            L.gqa_decode_blocks.restype = I
            L.gqa_decode_fp8kv_blocks.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, F, I, LP]
            L.gqa_decode_fp8kv_blocks.restype = I
            L.gqa_decode_blocks_plan_splits.argtypes = [I, I, I, I, I, I, I, I, I]
            L.gqa_decode_blocks_plan_splits.restype = I
            L.gqa_decode_weights.argtypes = [P, P, P, P, P, P, P, P, I, I, I, F, F, LP]
            L.gqa_decode_weights.restype = I
            L.gqa_decode_fp8kv_weights.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I, F, F, LP]
            L.gqa_decode_fp8kv_weights.restype = I
            L.gqa_decode_weights_workspace_size.argtypes = [I, I, I, I, I]
            L.gqa_decode_weights_workspace_size.restype = S
            L.gqa_decode_weights_plan_splits.argtypes = [I, I, I, I, I, I, I]
            L.gqa_decode_weights_plan_splits.restype = I
            L.gqa_block_bounds.argtypes = [P, P, P, P, P, I, I, I, LP]
            L.gqa_block_bounds.restype = I
            L.gqa_select_blocks.argtypes = [P, P, P, P, P, I, I, I, I, I, I, I, LP]
            L.gqa_select_blocks.restype = I
            L.gqa_select_workspace_size.argtypes = [I, I, I, I, I]
            L.gqa_select_workspace_size.restype = S
            L.gqa_kv_evict.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, LP]
            L.gqa_kv_evict.restype = I
            L.gqa_kv_append.argtypes = [P, P, P, P, P, P, I, I, LP]
            L.gqa_kv_append.restype = I
            L.gqa_kv_append_fp8kv.argtypes = [P, P, P, P, P, P, P, P, I, I, LP]
            L.gqa_kv_append_fp8kv.restype = I
            L.mla_kv_append.argtypes = [P, P, P, P, LP]
            L.mla_kv_append.restype = I
            L.mla_absorb_q.argtypes = [P, P, P, I, I, I, I, I, P, P]
            L.mla_absorb_q.restype = I
            L.mla_unabsorb_out.argtypes = [P, P, P, I, I, I, I, I, P, P]
            L.mla_unabsorb_out.restype = I
            L.mla_decode.argtypes = [P, P, P, P, P, P, F, LP]
            L.mla_decode.restype = I
            L.gqa_decode_plan_splits.argtypes = [I, I, I, I, I, I]
            L.gqa_decode_plan_splits.restype = I
            L.gqa_decode_fp8kv_plan_splits.argtypes = [I, I, I, I, I, I]
            L.gqa_decode_fp8kv_plan_splits.restype = I
            L.mla_decode_plan_splits.argtypes = [I, I, I]
            L.mla_decode_plan_splits.restype = I
            L.gqa_decode_workspace_size.argtypes = [I, I, I, I]
            L.gqa_decode_workspace_size.restype = S
            L.mla_decode_workspace_size.argtypes = [I, I]
            L.mla_decode_workspace_size.restype = S
            L.decattn_kv_bytes_per_token.argtypes = [I, I, I, I]
            L.decattn_kv_bytes_per_token.restype = I64
            L.decattn_mla_bytes_per_token.argtypes = [I, I, I, I]
            L.decattn_mla_bytes_per_token.restype = I64
            L.decattn_status_string.argtypes = [I]
            L.decattn_status_string.restype = ctypes.c_char_p
            L.decattn_selftest_wait_timeout.argtypes = [P, P, I, P]
            L.decattn_selftest_wait_timeout.restype = I
            L.decattn_selftest_warp_wait.argtypes = [P, P, I, P]
            L.decattn_selftest_warp_wait.restype = I
            L.decattn_selftest_gave_up.argtypes = [P, P, I, P]
            L.decattn_selftest_gave_up.restype = I
            L.decattn_version.argtypes = []
            L.decattn_version.restype = I
            _lib = L
    return _lib


def calls():
    """The native half of the binding (lib/_calls.so), opened on libdecattn.so."""
    global _calls
    if _calls is not None:
        return _calls
    lib()
    with _lock:
        if _calls is None:
            if not os.path.exists(_build.CALLS):
                raise RuntimeError(f"{_build.CALLS} is missing: build it with "
                                   "`python -m gqa_mqa_mla_gb300.build` (no fallback exists)")
            if not _build.calls_match():
                raise RuntimeError(f"{_build.CALLS} was built for another PyTorch: rebuild it with "
                                   "`python -m gqa_mqa_mla_gb300.build`")
            spec = importlib.util.spec_from_file_location("_calls", _build.CALLS)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            module.open(_build.LIB)
            _calls = module
    return _calls


def _decode_name(name: str, window, sinks: int) -> str:
    return name if window is None else name + ("_sinks" if sinks else "_window")


def selftest_warp_wait(limit_us: int = 1000, device="cuda"):
    """Run the self test of a warp's waits; returns (err_flag, result list of 4 ints)."""
    flag = torch.zeros(1, dtype=torch.int32, device=device)
    res = torch.full((4,), -1, dtype=torch.int32, device=device)
    st = lib().decattn_selftest_warp_wait(flag.data_ptr(), res.data_ptr(), int(limit_us),
                                          _stream_handle(None))
    if st != DECATTN_OK:
        raise DecAttnError("decattn_selftest_warp_wait", st)
    torch.cuda.synchronize()
    return int(flag.item()), res.tolist()


def selftest_gave_up(limit_us: int = 1000, device="cuda"):
    """Run the self test of a weighing decode's split that gives up; returns (err_flag,
    float tensor [40, 3]: a row's sums by split)."""
    flag = torch.zeros(1, dtype=torch.int32, device=device)
    res = torch.full((40, 3), -1.0, device=device)
    st = lib().decattn_selftest_gave_up(flag.data_ptr(), res.data_ptr(), int(limit_us),
                                        _stream_handle(None))
    if st != DECATTN_OK:
        raise DecAttnError("decattn_selftest_gave_up", st)
    torch.cuda.synchronize()
    return int(flag.item()), res.cpu()


def selftest_wait_timeout(limit_us: int = 1000, device="cuda"):
    """Run the bounded-wait self test; returns (err_flag, result list of 5 ints)."""
    flag = torch.zeros(1, dtype=torch.int32, device=device)
    res = torch.full((5,), -1, dtype=torch.int32, device=device)
    st = lib().decattn_selftest_wait_timeout(flag.data_ptr(), res.data_ptr(), int(limit_us),
                                              _stream_handle(None))
    if st != DECATTN_OK:
        raise DecAttnError("decattn_selftest_wait_timeout", st)
    torch.cuda.synchronize()
    return int(flag.item()), res.cpu().tolist()


def status_string(status: int) -> str:
    return lib().decattn_status_string(int(status)).decode()


def kv_bytes_per_token(n_layers: int, n_kv: int, d_head: int, bytes_per_elem: int) -> int:
    return int(lib().decattn_kv_bytes_per_token(n_layers, n_kv, d_head, bytes_per_elem))


def mla_bytes_per_token(n_layers: int, d_c: int, d_rope: int, bytes_per_elem: int) -> int:
    return int(lib().decattn_mla_bytes_per_token(n_layers, d_c, d_rope, bytes_per_elem))


def gqa_plan_splits(batch: int, h_q: int, h_kv: int, max_seq_len: int, d_head: int = 128,
                    num_sms: int = 0) -> int:
    r = lib().gqa_decode_plan_splits(batch, h_q, h_kv, d_head, max_seq_len, num_sms)
    if r < 0:
        raise DecAttnError("gqa_decode_plan_splits", r)
    return r


def gqa_fp8_plan_splits(batch: int, h_q: int, h_kv: int, max_seq_len: int, d_head: int = 128,
                        num_sms: int = 0) -> int:
    r = lib().gqa_decode_fp8kv_plan_splits(batch, h_q, h_kv, d_head, max_seq_len, num_sms)
    if r < 0:
        raise DecAttnError("gqa_decode_fp8kv_plan_splits", r)
    return r


def gqa_window_plan_splits(batch: int, h_q: int, h_kv: int, max_seq_len: int, window: int,
                           block_size: int, kv_bytes: int = 2, d_head: int = 128,
                           num_sms: int = 0) -> int:
    r = lib().gqa_decode_window_plan_splits(batch, h_q, h_kv, d_head, max_seq_len, window,
                                            block_size, kv_bytes, num_sms)
    if r < 0:
        raise DecAttnError("gqa_decode_window_plan_splits", r)
    return r


def gqa_sinks_plan_splits(batch: int, h_q: int, h_kv: int, max_seq_len: int, window: int,
                          sinks: int, block_size: int, kv_bytes: int = 2, d_head: int = 128,
                          num_sms: int = 0) -> int:
    r = lib().gqa_decode_sinks_plan_splits(batch, h_q, h_kv, d_head, max_seq_len, window, sinks,
                                           block_size, kv_bytes, num_sms)
    if r < 0:
        raise DecAttnError("gqa_decode_sinks_plan_splits", r)
    return r


def gqa_prefill_plan_splits(batch: int, tokens: int, max_q_len: int, h_q: int, h_kv: int,
                            max_seq_len: int, window: int = 0, sinks: int = 0, d_head: int = 128,
                            num_sms: int = 0) -> int:
    r = lib().gqa_prefill_plan_splits(batch, tokens, max_q_len, h_q, h_kv, d_head, max_seq_len,
                                      window, sinks, num_sms)
    if r < 0:
        raise DecAttnError("gqa_prefill_plan_splits", r)
    return r


def gqa_blocks_plan_splits(batch: int, h_q: int, h_kv: int, max_seq_len: int, count: int,
                           block_size: int, kv_bytes: int = 2, d_head: int = 128,
                           num_sms: int = 0) -> int:
    r = lib().gqa_decode_blocks_plan_splits(batch, h_q, h_kv, d_head, max_seq_len, count,
                                            block_size, kv_bytes, num_sms)
    if r < 0:
        raise DecAttnError("gqa_decode_blocks_plan_splits", r)
    return r


def gqa_weights_plan_splits(batch: int, h_q: int, h_kv: int, max_seq_len: int, kv_bytes: int = 2,
                            d_head: int = 128, num_sms: int = 0) -> int:
    r = lib().gqa_decode_weights_plan_splits(batch, h_q, h_kv, d_head, max_seq_len, kv_bytes,
                                             num_sms)
    if r < 0:
        raise DecAttnError("gqa_decode_weights_plan_splits", r)
    return r


def gqa_weights_workspace_size(batch: int, h_q: int, max_seq_len: int, num_splits: int,
                               d_head: int = 128) -> int:
    return int(lib().gqa_decode_weights_workspace_size(batch, h_q, d_head, max_seq_len,
                                                       num_splits))


def gqa_select_workspace_size(batch: int, h_kv: int, max_seq_len: int, block_size: int,
                              count: int) -> int:
    return int(lib().gqa_select_workspace_size(batch, h_kv, max_seq_len, block_size, count))


def gqa_prefill_workspace_size(tokens: int, h_q: int, num_splits: int, d_head: int = 128) -> int:
    return int(lib().gqa_prefill_workspace_size(tokens, h_q, d_head, num_splits))


def mla_plan_splits(batch: int, max_seq_len: int, num_sms: int = 0) -> int:
    r = lib().mla_decode_plan_splits(batch, max_seq_len, num_sms)
    if r < 0:
        raise DecAttnError("mla_decode_plan_splits", r)
    return r


def gqa_workspace_size(batch: int, h_q: int, num_splits: int, d_head: int = 128) -> int:
    return int(lib().gqa_decode_workspace_size(batch, h_q, d_head, num_splits))


def mla_workspace_size(batch: int, num_splits: int) -> int:
    return int(lib().mla_decode_workspace_size(batch, num_splits))


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _check(t: torch.Tensor, name: str, dtype=None, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name}: expected {ndim} dims, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_sinks(window, sinks):
    if sinks < 0:
        raise ValueError("sinks must not be negative")
    if sinks and window is None:
        raise ValueError("sinks need a window (without one every token is visible)")


def _window(window) -> int | None:
    return None if window is None else int(window)


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _handle(stream) -> int | None:
    """A given stream's handle; None stays: the native calls take the current
    stream of the tensors' device."""
    return None if stream is None else _stream_handle(stream)


def make_launch(batch, num_blocks, block_size, max_blocks_per_seq, max_seq_len, num_splits,
                dtype, workspace=None, workspace_bytes=0, err_flag=None, stream=None) -> Launch:
    return Launch(batch, num_blocks, block_size, max_blocks_per_seq, max_seq_len, num_splits,
                  dtype, workspace, workspace_bytes, err_flag, stream)


def _dense(t: torch.Tensor) -> bool:
    """No bytes between the tensor's elements, in whatever order its strides are."""
    n = 1
    for step, size in sorted((st, s) for s, st in zip(t.shape, t.stride()) if s != 1):
        if step != n:
            return False
        n *= size
    return True


class _CtypesCalls:
    """The GQA decode calls without the native half: the same arguments, checks and
    results, at some 10 us more a call."""

    @staticmethod
    def decode(q, kc, vc, k_scale, v_scale, table, lens, scale, max_seq_len, window, sinks,
               num_splits, out, workspace, err_flag, stream):
        fp8 = k_scale is not None
        _check(q, "q", ndim=3)
        if q.dtype not in _DT:
            raise TypeError("q must be float16 or bfloat16")
        for t, name in ((kc, "k_cache"), (vc, "v_cache")):
            codes = isinstance(t, torch.Tensor) and t.dtype == torch.float8_e4m3fn
            _check(t, name, q.dtype if not fp8 else t.dtype if codes else torch.uint8, 4)
        _check(table, "block_table", torch.int32, 2)
        _check(lens, "seq_lens", torch.int32, 1)
        B, h_q, d = q.shape
        nb, bs, h_kv, _ = kc.shape
        if kc.shape[3] != d or vc.shape != kc.shape:
            raise ValueError("k_cache / v_cache shape mismatch")
        if table.shape[0] < B or lens.shape[0] < B:
            raise ValueError(f"block_table and seq_lens need an entry for each of the {B} rows of q")
        if h_kv < 1 or h_q % h_kv != 0:
            raise ValueError(f"h_q={h_q} is not a multiple of h_kv={h_kv}")
        scales = [k_scale, v_scale] if fp8 else []
        for t in scales:
            _check(t, "k_scale / v_scale", torch.float32, 1)
            if t.shape[0] != h_kv:
                raise ValueError("k_scale / v_scale must be [h_kv]")
        if not q.is_cuda:
            raise ValueError("the tensors must be on a CUDA device")
        if out is not None:
            _check(out, "out", q.dtype)
            if out.numel() < q.numel():
                raise ValueError(f"out: expected shape {tuple(q.shape)}, got {tuple(out.shape)}")
        for t, name in ((workspace, "workspace"), (err_flag, "err_flag")):
            if t is not None and not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
        if workspace is not None and not _dense(workspace):
            raise ValueError("workspace must be dense")
        if err_flag is not None and err_flag.numel() * err_flag.element_size() < 4:
            raise ValueError("err_flag needs one int32 element")
        for t in (kc, vc, table, lens, *scales, out, workspace, err_flag):
            if t is not None and not (t.device == q.device or (not t.is_cuda and t.is_pinned())):
                raise ValueError(f"a tensor is on {t.device}, q on {q.device}")
        caller = torch.cuda.current_stream(q.device)
        if stream is None or stream == caller.cuda_stream:
            own = caller
        elif stream == 0:  # (ExternalStream takes 0 for "a new one")
            own = torch.cuda.default_stream(q.device)
        else:
            own = torch.cuda.ExternalStream(stream, device=q.device)
        L_ = lib()
        with torch.cuda.device(q.device), torch.cuda.stream(own):
            ns = num_splits
            if not ns:
                ns = L_.gqa_decode_sinks_plan_splits(B, h_q, h_kv, d, max_seq_len, window, sinks, bs,
                                                     1 if fp8 else 2, 0) if window is not None else \
                    (L_.gqa_decode_fp8kv_plan_splits if fp8 else L_.gqa_decode_plan_splits)(
                        B, h_q, h_kv, d, max_seq_len, 0)
                if ns < 0:
                    return ns
            if out is None:
                out = torch.empty_like(q)
                out.record_stream(caller)
            need = int(L_.gqa_decode_workspace_size(B, h_q, d, ns)) if ns > 1 else 0
            if need and workspace is None:
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
            size = 0 if workspace is None else workspace.numel() * workspace.element_size()
            L = make_launch(B, nb, bs, table.shape[1], max_seq_len, ns, _DT[q.dtype],
                            _ptr(workspace), size, _ptr(err_flag), own.cuda_stream)
            args = [t.data_ptr() for t in (q, kc, vc, *scales, table, lens, out)]
            args += [h_q, h_kv, d, float(scale)]
            if window is not None:
                args += [window] + ([sinks] if sinks else [])
            name = _decode_name("gqa_decode_fp8kv" if fp8 else "gqa_decode", window, sinks)
            st = getattr(L_, name)(*args, ctypes.byref(L))
        return out if st == DECATTN_OK else st


def _decode_calls():
    """The native calls; without them (not built, or for another PyTorch) ctypes."""
    if _calls is not None:
        return _calls
    lib()
    try:
        return calls()
    except (RuntimeError, ImportError) as e:
        warnings.warn(f"the GQA decode calls go through ctypes, some 10 us slower: {e}",
                      RuntimeWarning, stacklevel=3)
        return _CtypesCalls


def gqa_decode(q, k_cache, v_cache, block_table, seq_lens, *, scale: float, max_seq_len: int,
               out=None, num_splits: int = 0, workspace=None, err_flag=None, stream=None,
               window: int | None = None, sinks: int = 0):
    """MHA/GQA/MQA decode through the C ABI; returns out [B, h_q, d].

    q [B, h_q, d]; k_cache/v_cache [num_blocks, block_size, h_kv, d];
    block_table int32 [B, max_blocks]; seq_lens int32 [B] (either may have more
    entries: the first B count); max_seq_len a host upper bound of seq_lens.
    workspace: optional uint8 CUDA tensor (sized by gqa_workspace_size); allocated
    here when needed and not given.  window: attend only to each sequence's last
    `window` tokens (gqa_decode_window), and with sinks > 0 to its first `sinks`
    tokens too (gqa_decode_sinks).
    """
    _check_sinks(window, sinks)
    r = _decode_calls().decode(q, k_cache, v_cache, None, None, block_table, seq_lens, scale,
                               max_seq_len, _window(window), sinks, num_splits, out, workspace,
                               err_flag, _handle(stream))
    if type(r) is int:
        raise DecAttnError(_decode_name("gqa_decode", window, sinks), r)
    return r


def gqa_decode_sinks(q, k_cache, v_cache, block_table, seq_lens, *, window: int, sinks: int, **kw):
    """gqa_decode restricted to each sequence's first `sinks` and last `window` tokens."""
    return gqa_decode(q, k_cache, v_cache, block_table, seq_lens, window=window, sinks=sinks, **kw)


def gqa_decode_window(q, k_cache, v_cache, block_table, seq_lens, *, window: int, **kw):
    """gqa_decode restricted to each sequence's last `window` tokens."""
    return gqa_decode(q, k_cache, v_cache, block_table, seq_lens, window=window, **kw)


def gqa_decode_fp8kv(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens, *,
                     scale: float, max_seq_len: int, out=None, num_splits: int = 0,
                     workspace=None, err_flag=None, stream=None, window: int | None = None,
                     sinks: int = 0):
    """GQA decode over an 8-bit (e4m3) KV cache through the C ABI; returns out.

    q [B, h_q, d] fp16/bf16; k_codes/v_codes uint8 (or float8_e4m3fn)
    [num_blocks, block_size, h_kv, d]; k_scale/v_scale float32 [h_kv] (the
    value of KV head j is e4m3(code) * scale[j]); the rest as gqa_decode
    (window: gqa_decode_fp8kv_window; sinks: gqa_decode_fp8kv_sinks).
    """
    _check_sinks(window, sinks)
    if k_scale is None or v_scale is None:
        raise TypeError("k_scale and v_scale must be torch.Tensors")
    r = _decode_calls().decode(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens, scale,
                               max_seq_len, _window(window), sinks, num_splits, out, workspace,
                               err_flag, _handle(stream))
    if type(r) is int:
        raise DecAttnError(_decode_name("gqa_decode_fp8kv", window, sinks), r)
    return r


def gqa_decode_fp8kv_window(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens, *,
                            window: int, **kw):
    """gqa_decode_fp8kv restricted to each sequence's last `window` tokens."""
    return gqa_decode_fp8kv(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens,
                            window=window, **kw)


def gqa_decode_fp8kv_sinks(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens, *,
                           window: int, sinks: int, **kw):
    """gqa_decode_fp8kv restricted to each sequence's first `sinks` and last `window` tokens."""
    return gqa_decode_fp8kv(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens,
                            window=window, sinks=sinks, **kw)


def _append_launch(new, cache, block_table, dtype, err_flag, stream) -> Launch:
    return make_launch(new.shape[0], cache.shape[0], cache.shape[1], block_table.shape[1], 0, 1,
                       _DT[dtype], None, 0, _ptr(err_flag), _stream_handle(stream))


def gqa_kv_append(k_new, v_new, positions, block_table, k_cache, v_cache, *, err_flag=None,
                  stream=None):
    """Write each sequence's new K/V rows [B, h_kv, d] into slot positions[b]
    of its paged 16-bit cache (in place); a negative position skips."""
    _check(k_new, "k_new", ndim=3)
    _check(v_new, "v_new", k_new.dtype, 3)
    _check(k_cache, "k_cache", k_new.dtype, 4)
    _check(v_cache, "v_cache", k_new.dtype, 4)
    _check(positions, "positions", torch.int32, 1)
    _check(block_table, "block_table", torch.int32, 2)
    if k_new.dtype not in _DT:
        raise TypeError("k_new must be float16 or bfloat16")
    B, h_kv, d = k_new.shape
    if v_new.shape != k_new.shape or k_cache.shape[2:] != (h_kv, d) or \
            v_cache.shape != k_cache.shape or positions.shape != (B,) or block_table.shape[0] != B:
        raise ValueError("kv_append: shape mismatch")
    L = _append_launch(k_new, k_cache, block_table, k_new.dtype, err_flag, stream)
    st = lib().gqa_kv_append(k_new.data_ptr(), v_new.data_ptr(), positions.data_ptr(),
                             block_table.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), h_kv,
                             d, ctypes.byref(L))
    if st != DECATTN_OK:
        raise DecAttnError("gqa_kv_append", st)


def gqa_kv_append_fp8kv(k_new, v_new, k_scale, v_scale, positions, block_table, k_codes, v_codes,
                        *, err_flag=None, stream=None):
    """Quantise each sequence's new K/V rows [B, h_kv, d] (fp16/bf16) to e4m3
    codes with the per-KV-head scales and write them into slot positions[b]
    of the 8-bit cache (uint8 or float8_e4m3fn, in place)."""
    if k_codes.dtype == torch.float8_e4m3fn:
        k_codes = k_codes.view(torch.uint8)
    if v_codes.dtype == torch.float8_e4m3fn:
        v_codes = v_codes.view(torch.uint8)
    _check(k_new, "k_new", ndim=3)
    _check(v_new, "v_new", k_new.dtype, 3)
    _check(k_scale, "k_scale", torch.float32, 1)
    _check(v_scale, "v_scale", torch.float32, 1)
    _check(k_codes, "k_codes", torch.uint8, 4)
    _check(v_codes, "v_codes", torch.uint8, 4)
    _check(positions, "positions", torch.int32, 1)
    _check(block_table, "block_table", torch.int32, 2)
    if k_new.dtype not in _DT:
        raise TypeError("k_new must be float16 or bfloat16")
    B, h_kv, d = k_new.shape
    if v_new.shape != k_new.shape or k_codes.shape[2:] != (h_kv, d) or \
            v_codes.shape != k_codes.shape or positions.shape != (B,) or \
            block_table.shape[0] != B or k_scale.shape != (h_kv,) or v_scale.shape != (h_kv,):
        raise ValueError("kv_append_fp8kv: shape mismatch")
    L = _append_launch(k_new, k_codes, block_table, k_new.dtype, err_flag, stream)
    st = lib().gqa_kv_append_fp8kv(k_new.data_ptr(), v_new.data_ptr(), k_scale.data_ptr(),
                                   v_scale.data_ptr(), positions.data_ptr(),
                                   block_table.data_ptr(), k_codes.data_ptr(), v_codes.data_ptr(),
                                   h_kv, d, ctypes.byref(L))
    if st != DECATTN_OK:
        raise DecAttnError("gqa_kv_append_fp8kv", st)


def paged_plan(cached_lens, new_lens, block_table, free_blocks, free_count, *, block_size: int,
               max_tokens: int, seq_lens=None, q_start=None, slots=None, positions=None,
               free_count_out=None, err_flag=None, stream=None) -> PagedPlan:
    """A serving step's paged state from the requests' lengths, on the GPU.

    cached_lens, new_lens int32 [B] (new < 0 gives tokens back); block_table
    int32 [B, max_blocks] and free_blocks int32 [num_blocks] (a stack of
    free_count[0] ids) are updated in place.  The outputs are allocated when
    not given, as parts of one storage (a kept seq_lens keeps that step's slots
    and positions in memory too); free_count_out may be free_count and seq_lens may
    be cached_lens (in place).  Rows past the step's last token get slot and
    position -1.
    """
    r = calls().paged_plan(cached_lens, new_lens, block_table, free_blocks, free_count, block_size,
                           max_tokens, seq_lens, q_start, slots, positions, free_count_out,
                           err_flag, _handle(stream))
    if type(r) is int:
        raise DecAttnError("paged_plan", r)
    return PagedPlan(*r)


def rope_table(inv_freq, *, sections=None, interleaved: bool = False, device=None) -> RopeTable:
    """How a model's heads are rotated, for gqa_rope_append.

    inv_freq: rot_dim / 2 frequencies (radians per position), a sequence or a
    tensor; sections: how many consecutive pairs follow each position axis
    (default: one axis); interleaved: pairs (2 i, 2 i + 1) instead of
    (i, i + rot_dim / 2).  Host data (`device` is accepted for symmetry with
    tensor factories and ignored).
    """
    freq = [float(f) for f in (inv_freq.tolist() if isinstance(inv_freq, torch.Tensor)
                               else inv_freq)]
    cut = None if sections is None else [int(n) for n in sections]
    rope = RopeTable()
    st = lib().decattn_rope_fill(
        ctypes.byref(rope), (ctypes.c_double * max(1, len(freq)))(*freq), 2 * len(freq),
        None if cut is None else (ctypes.c_int * max(1, len(cut)))(*cut),
        1 if cut is None else len(cut), int(bool(interleaved)))
    if st != DECATTN_OK:
        raise DecAttnError("decattn_rope_fill", st)
    return rope


def _rope_append(name, q, k_new, v_new, k_scale, v_scale, positions, rope, slots, k_cache, v_cache,
                 q_out, err_flag, stream):
    if not isinstance(rope, RopeTable):
        raise TypeError("rope must come from rope_table")
    r = calls().rope_append(q, k_new, v_new, k_scale, v_scale, positions, ctypes.addressof(rope),
                            rope.n_axes, slots, k_cache, v_cache, q_out, err_flag, _handle(stream))
    if type(r) is int:
        raise DecAttnError(name, r)
    return r


def gqa_rope_append(q, k_new, v_new, positions, rope, slots, k_cache, v_cache, *, q_out=None,
                    err_flag=None, stream=None):
    """Rotate q and k by their positions, write k and v into the paged cache's
    slots (in place) and return the rotated q [T, h_q, d].

    q [T, h_q, d], k_new / v_new [T, h_kv, d]: each token's heads contiguous,
    tokens any stride (parts of one projection's output); positions int32
    [n_axes, T] (or [T]); rope: rope_table's; slots int32 [T] (negative: no
    cache row); q_out: a contiguous [T, h_q, d], may be q.
    """
    return _rope_append("gqa_rope_append", q, k_new, v_new, None, None, positions, rope, slots,
                        k_cache, v_cache, q_out, err_flag, stream)


def gqa_rope_append_fp8kv(q, k_new, v_new, k_scale, v_scale, positions, rope, slots, k_codes,
                          v_codes, *, q_out=None, err_flag=None, stream=None):
    """gqa_rope_append into an 8-bit e4m3 cache (uint8 or float8_e4m3fn) with
    one scale per KV head."""
    if k_scale is None or v_scale is None:
        raise TypeError("k_scale and v_scale must be torch.Tensors")
    return _rope_append("gqa_rope_append_fp8kv", q, k_new, v_new, k_scale, v_scale, positions, rope,
                        slots, k_codes, v_codes, q_out, err_flag, stream)


def _prefill(name, q, k_cache, v_cache, k_scale, v_scale, block_table, q_start, seq_lens, scale,
             max_q_len, max_seq_len, window, sinks, out, num_splits, workspace, err_flag, stream):
    _check_sinks(window, sinks)
    if window is not None and window < 1:
        raise ValueError("window must be at least 1")
    r = calls().prefill(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, q_start,
                        scale, max_q_len, max_seq_len, window or 0, sinks, num_splits, out,
                        workspace, err_flag, _handle(stream))
    if type(r) is int:
        raise DecAttnError(name, r)
    return r


def gqa_prefill(q, k_cache, v_cache, block_table, q_start, seq_lens, *, scale: float,
                max_q_len: int, max_seq_len: int, window: int | None = None, sinks: int = 0,
                out=None, num_splits: int = 0, workspace=None, err_flag=None, stream=None):
    """Attention of a chunk of new tokens per sequence over the paged cache;
    returns out [T, h_q, d].

    q [T, h_q, d] packed rows, sequence b's being q_start[b] .. q_start[b + 1]
    - 1 (int32 [B + 1]); seq_lens int32 [B] counts the cached tokens, the
    chunk included; row i of a chunk of n is position seq_lens[b] - n + i and
    sees the positions up to its own, of them the last `window` and the first
    `sinks` where a window is given.  max_q_len, max_seq_len: host upper
    bounds.  Rows outside every sequence are not written.
    """
    return _prefill("gqa_prefill", q, k_cache, v_cache, None, None, block_table, q_start, seq_lens,
                    scale, max_q_len, max_seq_len, window, sinks, out, num_splits, workspace,
                    err_flag, stream)


def gqa_prefill_fp8kv(q, k_codes, v_codes, k_scale, v_scale, block_table, q_start, seq_lens, *,
                      scale: float, max_q_len: int, max_seq_len: int, window: int | None = None,
                      sinks: int = 0, out=None, num_splits: int = 0, workspace=None,
                      err_flag=None, stream=None):
    """gqa_prefill over an 8-bit e4m3 cache (uint8 or float8_e4m3fn) with one
    scale per KV head."""
    if k_scale is None or v_scale is None:
        raise TypeError("k_scale and v_scale must be torch.Tensors")
    return _prefill("gqa_prefill_fp8kv", q, k_codes, v_codes, k_scale, v_scale, block_table, q_start,
                    seq_lens, scale, max_q_len, max_seq_len, window, sinks, out, num_splits,
                    workspace, err_flag, stream)


def gqa_block_bounds(k_cache, block_table, seq_lens, bounds, *, max_seq_len: int, first_lens=None,
                     err_flag=None, stream=None):
    """Smallest and largest key of cache blocks, per KV head and dimension, for
    gqa_select_blocks; updates bounds [num_blocks, 2, h_kv, d] in place and returns it.

    k_cache [num_blocks, block_size, h_kv, d] fp16/bf16, or e4m3 codes (uint8 or
    float8_e4m3fn); bounds of the same type; block_table int32 [B, max_blocks],
    seq_lens int32 [B].  first_lens int32 [B]: the tokens whose blocks are up to
    date (each sequence's length before the step); without it every block is taken.
    """
    r = calls().block_bounds(k_cache, block_table, seq_lens, bounds, first_lens, max_seq_len,
                             err_flag, _handle(stream))
    if type(r) is int:
        raise DecAttnError("gqa_block_bounds", r)
    return r


def gqa_select_blocks(q, bounds, block_table, seq_lens, *, block_size: int, max_seq_len: int,
                      count: int, first: int = 1, last: int = 1, out=None, workspace=None,
                      err_flag=None, stream=None):
    """The `count` blocks of each sequence that can matter most to its query, per KV
    head; returns int32 [B, h_kv, count], block numbers within the sequence,
    ascending, -1 behind the last.

    q [B, h_q, d] fp16/bf16; bounds: gqa_block_bounds' (16-bit: q's type; or e4m3
    codes).  The sequence's `first` first and `last` last blocks are always among
    them, the others by the largest bound of q . k over their keys.  workspace:
    optional uint8 CUDA tensor (gqa_select_workspace_size bytes).
    """
    r = calls().select_blocks(q, bounds, block_table, seq_lens, block_size, max_seq_len, count,
                              first, last, out, workspace, err_flag, _handle(stream))
    if type(r) is int:
        raise DecAttnError("gqa_select_blocks", r)
    return r


def gqa_decode_blocks(q, k_cache, v_cache, block_table, seq_lens, selected, *, scale: float,
                      max_seq_len: int, out=None, num_splits: int = 0, workspace=None,
                      err_flag=None, stream=None):
    """gqa_decode over the blocks that selected [B, h_kv, count] (int32, ascending
    block numbers within the sequence, -1 behind the last: gqa_select_blocks') lists
    for each sequence and KV head; returns out [B, h_q, d]."""
    r = calls().decode_blocks(q, k_cache, v_cache, None, None, block_table, seq_lens, selected,
                              scale, max_seq_len, num_splits, out, workspace, err_flag,
                              _handle(stream))
    if type(r) is int:
        raise DecAttnError("gqa_decode_blocks", r)
    return r


def gqa_decode_fp8kv_blocks(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens,
                            selected, *, scale: float, max_seq_len: int, out=None,
                            num_splits: int = 0, workspace=None, err_flag=None, stream=None):
    """gqa_decode_blocks over an 8-bit e4m3 cache (uint8 or float8_e4m3fn) with one
    scale per KV head."""
    if k_scale is None or v_scale is None:
        raise TypeError("k_scale and v_scale must be torch.Tensors")
    r = calls().decode_blocks(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens,
                              selected, scale, max_seq_len, num_splits, out, workspace, err_flag,
                              _handle(stream))
    if type(r) is int:
        raise DecAttnError("gqa_decode_fp8kv_blocks", r)
    return r


def gqa_decode_weights(q, k_cache, v_cache, weights, block_table, seq_lens, *, scale: float,
                       max_seq_len: int, weighed_lens=None, decay: float = 1.0, out=None,
                       num_splits: int = 0, workspace=None, err_flag=None, stream=None):
    """gqa_decode that adds up each cached token's attention weight; returns out.

    weights float32 [num_blocks, h_kv, block_size], updated in place: the slot of
    each token t < seq_lens[b] gets (decay times its old value where t <
    weighed_lens[b], else 0) plus the softmax weights that the KV head's query heads
    give it.  weighed_lens int32 [B]: the tokens that have weights already (after a
    prompt, 0: its slots hold what their blocks' last user left); without it all but
    the last.  workspace: gqa_weights_workspace_size bytes.
    """
    r = calls().decode_weights(q, k_cache, v_cache, None, None, block_table, seq_lens, weights,
                               weighed_lens, scale, decay, max_seq_len, num_splits, out, workspace,
                               err_flag, _handle(stream))
    if type(r) is int:
        raise DecAttnError("gqa_decode_weights", r)
    return r


def gqa_decode_fp8kv_weights(q, k_codes, v_codes, k_scale, v_scale, weights, block_table,
                             seq_lens, *, scale: float, max_seq_len: int, weighed_lens=None,
                             decay: float = 1.0, out=None, num_splits: int = 0, workspace=None,
                             err_flag=None, stream=None):
    """gqa_decode_weights over an 8-bit e4m3 cache (uint8 or float8_e4m3fn) with one
    scale per KV head."""
    if k_scale is None or v_scale is None:
        raise TypeError("k_scale and v_scale must be torch.Tensors")
    r = calls().decode_weights(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens,
                               weights, weighed_lens, scale, decay, max_seq_len, num_splits, out,
                               workspace, err_flag, _handle(stream))
    if type(r) is int:
        raise DecAttnError("gqa_decode_fp8kv_weights", r)
    return r


def gqa_kv_evict(k_cache, v_cache, weights, block_table, seq_lens, *, max_seq_len: int, keep: int,
                 recent: int, limit: int | None = None, new_lens=None, kept=None, err_flag=None,
                 stream=None) -> Evicted:
    """Sequences longer than `limit` (default: keep) go back to `keep` tokens: per KV
    head the last `recent` and the heaviest others by weights (gqa_decode_weights'),
    moved in order to the sequence's front.

    k_cache, v_cache (fp16/bf16, or e4m3 codes as uint8 or float8_e4m3fn) and
    weights are updated in place.  Returns new_lens [B] (minus the tokens evicted:
    paged_plan's new_lens, which frees their blocks) and kept [B, h_kv, keep] (the
    kept tokens' old positions, -1 where nothing is evicted).

    Afterwards the caller takes the sequences' bounds anew (gqa_block_bounds without
    first_lens), and adds the tokens evicted so far to paged_plan's positions, which
    count the tokens in the cache: kept keys carry the rotation of the positions that
    they had.
    """
    r = calls().kv_evict(k_cache, v_cache, weights, block_table, seq_lens, max_seq_len, keep,
                         recent, keep if limit is None else limit, new_lens, kept, err_flag,
                         _handle(stream))
    if type(r) is int:
        raise DecAttnError("gqa_kv_evict", r)
    return Evicted(*r)


def mla_kv_append(latent_new, positions, block_table, latent_cache, *, err_flag=None,
                  stream=None):
    """Write each sequence's new latent row [B, 576] (c_t then the RoPE key)
    into slot positions[b] of the paged latent cache (in place)."""
    _check(latent_new, "latent_new", ndim=2)
    _check(latent_cache, "latent_cache", latent_new.dtype, 3)
    _check(positions, "positions", torch.int32, 1)
    _check(block_table, "block_table", torch.int32, 2)
    if latent_new.dtype not in _DT:
        raise TypeError("latent_new must be float16 or bfloat16")
    B = latent_new.shape[0]
    if latent_new.shape[1] != 576 or latent_cache.shape[2] != 576 or positions.shape != (B,) or \
            block_table.shape[0] != B:
        raise ValueError("mla_kv_append: shape mismatch")
    L = _append_launch(latent_new, latent_cache, block_table, latent_new.dtype, err_flag, stream)
    st = lib().mla_kv_append(latent_new.data_ptr(), positions.data_ptr(), block_table.data_ptr(),
                             latent_cache.data_ptr(), ctypes.byref(L))
    if st != DECATTN_OK:
        raise DecAttnError("mla_kv_append", st)


def mla_absorb_q(q_nope, w_uk, *, out=None, err_flag=None, stream=None):
    """q_abs[b, i, :] = q_nope[b, i, :] W_uk^(i)^T through the C ABI.

    q_nope [B, H, d_h]; w_uk [H, d_c, d_h] (w_uk[i] = W_uk^(i)); returns
    q_abs [B, H, d_c], mla_decode's absorbed query.
    """
    _check(q_nope, "q_nope", ndim=3)
    _check(w_uk, "w_uk", q_nope.dtype, 3)
    if q_nope.dtype not in _DT:
        raise TypeError("q_nope must be float16 or bfloat16")
    B, H, d_h = q_nope.shape
    if w_uk.shape[0] != H or w_uk.shape[2] != d_h:
        raise ValueError("w_uk must be [H, d_c, d_h]")
    d_c = w_uk.shape[1]
    if out is None:
        out = torch.empty((B, H, d_c), dtype=q_nope.dtype, device=q_nope.device)
    _check(out, "out", q_nope.dtype, 3)
    st = lib().mla_absorb_q(q_nope.data_ptr(), w_uk.data_ptr(), out.data_ptr(), B, H, d_h, d_c,
                            _DT[q_nope.dtype], _ptr(err_flag), _stream_handle(stream))
    if st != DECATTN_OK:
        raise DecAttnError("mla_absorb_q", st)
    return out


def mla_unabsorb_out(o_lat, w_uv_t, *, out=None, err_flag=None, stream=None):
    """out[b, i, :] = o_lat[b, i, :] W_uv^(i) through the C ABI.

    o_lat [B, H, d_c] (mla_decode's output); w_uv_t [H, d_v, d_c] (w_uv_t[i]
    = W_uv^(i) transposed); returns [B, H, d_v].
    """
    _check(o_lat, "o_lat", ndim=3)
    _check(w_uv_t, "w_uv_t", o_lat.dtype, 3)
    if o_lat.dtype not in _DT:
        raise TypeError("o_lat must be float16 or bfloat16")
    B, H, d_c = o_lat.shape
    if w_uv_t.shape[0] != H or w_uv_t.shape[2] != d_c:
        raise ValueError("w_uv_t must be [H, d_v, d_c]")
    d_v = w_uv_t.shape[1]
    if out is None:
        out = torch.empty((B, H, d_v), dtype=o_lat.dtype, device=o_lat.device)
    _check(out, "out", o_lat.dtype, 3)
    st = lib().mla_unabsorb_out(o_lat.data_ptr(), w_uv_t.data_ptr(), out.data_ptr(), B, H, d_c,
                                d_v, _DT[o_lat.dtype], _ptr(err_flag), _stream_handle(stream))
    if st != DECATTN_OK:
        raise DecAttnError("mla_unabsorb_out", st)
    return out


def mla_decode(q_absorbed, q_rope, latent_cache, block_table, seq_lens, *, scale: float,
               max_seq_len: int, out=None, num_splits: int = 0, workspace=None, err_flag=None,
               stream=None):
    """Absorbed MLA decode through the C ABI; returns out [B, 128, 512]."""
    _check(q_absorbed, "q_absorbed", ndim=3)
    _check(q_rope, "q_rope", q_absorbed.dtype, 3)
    _check(latent_cache, "latent_cache", q_absorbed.dtype, 3)
    _check(block_table, "block_table", torch.int32, 2)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    if q_absorbed.dtype not in _DT:
        raise TypeError("q_absorbed must be float16 or bfloat16")
    B = q_absorbed.shape[0]
    if q_absorbed.shape != (B, MLA_HEADS, MLA_D_C) or q_rope.shape != (B, MLA_HEADS, MLA_D_R):
        raise ValueError("q_absorbed must be [B,128,512] and q_rope [B,128,64]")
    nb, bs, width = latent_cache.shape
    if width != MLA_D_C + MLA_D_R:
        raise ValueError("latent_cache must be [num_blocks, block_size, 576]")
    if block_table.shape[0] < B or seq_lens.shape[0] < B:
        raise ValueError(f"block_table and seq_lens need an entry for each of the {B} rows of q")
    if out is None:
        out = torch.empty_like(q_absorbed)
    ns = num_splits if num_splits else mla_plan_splits(B, max_seq_len)
    need = mla_workspace_size(B, ns)
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q_absorbed.device)
    L = make_launch(B, nb, bs, block_table.shape[1], max_seq_len, ns, _DT[q_absorbed.dtype],
                    _ptr(workspace), 0 if workspace is None else workspace.numel(),
                    _ptr(err_flag), _stream_handle(stream))
    st = lib().mla_decode(q_absorbed.data_ptr(), q_rope.data_ptr(), latent_cache.data_ptr(),
                          block_table.data_ptr(), seq_lens.data_ptr(), out.data_ptr(),
                          float(scale), ctypes.byref(L))
    if st != DECATTN_OK:
        raise DecAttnError("mla_decode", st)
    return out
