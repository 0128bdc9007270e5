"""GB300 (sm_103a) fused exact attention: thin Python binding over libfa.so.

Every computation runs in the library's CUDA kernels; this module only checks
tensor properties, allocates outputs with torch and passes raw pointers plus the
current CUDA stream through the C ABI declared in ``include/fa.h`` (the packed and
cache calls do so in a compiled module, csrc/binding.cpp).  There is no
CPU or eager fallback: if the library is missing or a tensor is not a
contiguous bf16 CUDA tensor, the call raises.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch
from torch.autograd.function import once_differentiable

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfa.so")

FA_OK = 0
FA_ERR_WORKSPACE = 4
FA_ERR_TIMEOUT = 6
STATUS_NAMES = {0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED",
                3: "FA_ERR_MISALIGNED", 4: "FA_ERR_WORKSPACE", 5: "FA_ERR_CUDA",
                6: "FA_ERR_TIMEOUT"}

#: every symbol include/fa.h declares
EXPORTS = ("fa_fwd", "fa_fwd_status", "fa_bwd_workspace_bytes", "fa_bwd", "fa_bwd_status",
           "fa_status_string", "fa_exp2_test", "fa_last_launch_count", "fa_set_timing_events",
           "fa_set_bwd_kernel",
           "fa_bwd_noalloc", "fa_fwd_mod", "fa_bwd_mod", "fa_fwd_split_count",
           "fa_fwd_split_workspace_bytes", "fa_fwd_split", "fa_lse_merge", "fa_wait_test",
           "fa_bwd_noalloc_status", "fa_varlen_workspace_bytes", "fa_fwd_varlen",
           "fa_bwd_varlen", "fa_varlen_sink_workspace_bytes", "fa_fwd_varlen_sink",
           "fa_bwd_varlen_sink", "fa_cache4_page_bytes", "fa_cache4_append", "fa_cache4_read",
           "fa_cache4_attend_workspace_bytes", "fa_cache4_attend", "fa_cache4_evict",
           "fa_cache4_status", "fa_cache4_attend_sink", "fa_cache4_append_slots",
           "fa_page_update", "fa_norm_rope_fwd", "fa_norm_rope_bwd",
           "fa_norm_rope_workspace_bytes", "fa_rope_table")


class ScoreMod(ctypes.Structure):
    """fa_score_mod: a sliding window (negative sides unbounded), optional
    per-head relative-position bias slopes and optional per-batch key counts
    (device pointers or None)."""
    _fields_ = [("window_left", ctypes.c_int), ("window_right", ctypes.c_int),
                ("alibi_slopes", ctypes.c_void_p), ("seqlens_k", ctypes.c_void_p)]


class PackedStride(ctypes.Structure):
    """fa_packed_stride: elements from one token, and from one head, to the next."""
    _fields_ = [("token", ctypes.c_int64), ("head", ctypes.c_int64)]


_LIB = None


class FAError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(code, code)}")
        self.code = code


def _bind(lib):
    vp, i, f, sz, i64 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t,
                         ctypes.c_int64)
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp]
    lib.fa_fwd.restype = i
    lib.fa_fwd_status.argtypes = [vp]
    lib.fa_fwd_status.restype = i
    lib.fa_bwd_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    lib.fa_bwd_workspace_bytes.restype = sz
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, vp, sz, i,
                           vp]
    lib.fa_bwd.restype = i
    lib.fa_bwd_status.argtypes = [vp, vp]
    lib.fa_bwd_status.restype = i
    lib.fa_status_string.argtypes = [i]
    lib.fa_status_string.restype = ctypes.c_char_p
    lib.fa_exp2_test.argtypes = [vp, vp, i64, i, vp]
    lib.fa_exp2_test.restype = i
    lib.fa_last_launch_count.argtypes = []
    lib.fa_last_launch_count.restype = i
    lib.fa_set_timing_events.argtypes = [vp, vp]
    lib.fa_set_timing_events.restype = i
    lib.fa_set_bwd_kernel.argtypes = [i, vp]
    lib.fa_set_bwd_kernel.restype = i
    lib.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i,
                                   vp]
    lib.fa_bwd_noalloc.restype = i
    lib.fa_bwd_noalloc_status.argtypes = [vp]
    lib.fa_bwd_noalloc_status.restype = i
    smp = ctypes.POINTER(ScoreMod)
    lib.fa_fwd_mod.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, smp, f, vp]
    lib.fa_fwd_mod.restype = i
    lib.fa_bwd_mod.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, smp, f, vp,
                               sz, i, vp]
    lib.fa_bwd_mod.restype = i
    lib.fa_fwd_split_count.argtypes = [i, i, i, i, i]
    lib.fa_fwd_split_count.restype = i
    lib.fa_fwd_split_workspace_bytes.argtypes = [i, i, i, i, i, i]
    lib.fa_fwd_split_workspace_bytes.restype = sz
    lib.fa_fwd_split.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, smp, f, i, vp, sz, vp]
    lib.fa_fwd_split.restype = i
    lib.fa_lse_merge.argtypes = [vp, vp, i, vp, vp, i64, i, vp]
    lib.fa_lse_merge.restype = i
    lib.fa_wait_test.argtypes = [vp, i, vp, vp]
    lib.fa_wait_test.restype = i
    psp = ctypes.POINTER(PackedStride)
    lib.fa_varlen_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
    lib.fa_varlen_workspace_bytes.restype = sz
    lib.fa_fwd_varlen.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, psp, psp, psp, i, i, f,
                                  vp, sz, vp]
    lib.fa_fwd_varlen.restype = i
    lib.fa_bwd_varlen.argtypes = [vp] * 10 + [i, i, i, i, i, psp, psp, psp, i, i, f, vp, sz, i, vp]
    lib.fa_bwd_varlen.restype = i
    lib.fa_varlen_sink_workspace_bytes.argtypes = [i] * 9
    lib.fa_varlen_sink_workspace_bytes.restype = sz
    lib.fa_fwd_varlen_sink.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, psp, psp, psp, i, i,
                                       i, f, vp, sz, vp]
    lib.fa_fwd_varlen_sink.restype = i
    lib.fa_bwd_varlen_sink.argtypes = [vp] * 10 + [i, i, i, i, i, psp, psp, psp, i, i, i, f, vp,
                                                   sz, i, vp]
    lib.fa_bwd_varlen_sink.restype = i
    lib.fa_cache4_page_bytes.argtypes = [i, i, i]
    lib.fa_cache4_page_bytes.restype = sz
    lib.fa_cache4_append.argtypes = [vp, i, i, vp, vp, psp, psp, i, i, i, i, vp, vp, vp, i, vp]
    lib.fa_cache4_append.restype = i
    lib.fa_cache4_read.argtypes = [vp, i, i, vp, vp, i, i, i, i, vp, vp, vp, i, vp]
    lib.fa_cache4_read.restype = i
    lib.fa_cache4_attend_workspace_bytes.argtypes = [i, i, i, i, i]
    lib.fa_cache4_attend_workspace_bytes.restype = sz
    lib.fa_cache4_attend.argtypes = [vp, i64, i64, vp, i, i, vp, vp, i, i, i, i, vp, vp, i, f, vp,
                                     vp, i, vp, sz, vp]
    lib.fa_cache4_attend.restype = i
    lib.fa_cache4_attend_sink.argtypes = [vp, i64, i64, vp, i, i, vp, vp, i, i, i, i, vp, vp, i, i,
                                          i, f, vp, vp, i, vp, sz, vp]
    lib.fa_cache4_attend_sink.restype = i
    lib.fa_cache4_append_slots.argtypes = [vp, i, i, vp, vp, psp, psp, i, i, i, vp, vp]
    lib.fa_cache4_append_slots.restype = i
    lib.fa_page_update.argtypes = [vp, i, vp, vp, i, vp, vp, i, i, i, i, i, vp, vp, vp, vp]
    lib.fa_page_update.restype = i
    lib.fa_norm_rope_fwd.argtypes = [vp] * 6 + [i, vp, vp, vp, i, i, i, i, i, i, i, f, psp, psp, psp,
                                                psp, i, vp]
    lib.fa_norm_rope_fwd.restype = i
    lib.fa_norm_rope_workspace_bytes.argtypes = [i, i, i, i]
    lib.fa_norm_rope_workspace_bytes.restype = sz
    lib.fa_norm_rope_bwd.argtypes = [vp] * 10 + [i, vp, vp, vp, i, i, i, i, i, i, i, f, psp, psp,
                                                 psp, psp, psp, psp, i, vp, sz, vp]
    lib.fa_norm_rope_bwd.restype = i
    lib.fa_rope_table.argtypes = [vp, vp, i64, i, ctypes.c_double, vp]
    lib.fa_rope_table.restype = i
    lib.fa_cache4_evict.argtypes = [vp, i, i, vp, i, vp, vp, i, i, i, i, i, i, vp, i, vp, vp, vp,
                                    vp]
    lib.fa_cache4_evict.restype = i
    lib.fa_cache4_status.argtypes = [vp]
    lib.fa_cache4_status.restype = i
    return lib


def _score_mod(causal, window, alibi_slopes, Hq, seqlens_k=None, B=None):
    """The fa_score_mod for a call, or None when the plain entry point applies."""
    if window is None and alibi_slopes is None and seqlens_k is None:
        return None
    wl, wr = (-1, 0 if causal else -1) if window is None else window
    if causal and window is not None:
        raise ValueError("give the causal mask as window=(-1, 0), not with causal=True")
    ptr = None
    if alibi_slopes is not None:
        if (not alibi_slopes.is_cuda or alibi_slopes.dtype != torch.float32
                or alibi_slopes.numel() != Hq or not alibi_slopes.is_contiguous()):
            raise TypeError("alibi_slopes must be a contiguous fp32 CUDA tensor of Hq slopes")
        ptr = alibi_slopes.data_ptr()
    lens = None
    if seqlens_k is not None:
        if (not seqlens_k.is_cuda or seqlens_k.dtype != torch.int32
                or seqlens_k.numel() != B or not seqlens_k.is_contiguous()):
            raise TypeError("seqlens_k must be a contiguous int32 CUDA tensor of B key counts")
        lens = seqlens_k.data_ptr()
    # (a ctypes int would wrap; distances stay below 2^31)
    wl, wr = (max(-1, min(int(w), 2 ** 31 - 1)) for w in (wl, wr))
    return ScoreMod(wl, wr, ptr, lens)


def lib():
    """The loaded libfa.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build()")
        _LIB = _bind(ctypes.CDLL(LIB_PATH))
    return _LIB


def build(force: bool = False) -> str:
    from . import _build
    return _build.build(force=force)


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _new(shape, dtype, device, stream=None, returned=True):
    """New memory for a call on ``stream``: from that stream's pool, where nothing
    queued elsewhere still uses it.  What is returned stays until the caller's
    current stream, where it is used next, has passed."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _check(t: torch.Tensor, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous [B, H, S, D]")
    if t.dim() != 4:
        raise ValueError(f"{name} must be 4-D [B, H, S, D]")


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
        scale: float | None = None, out: torch.Tensor | None = None,
        lse: torch.Tensor | None = None, stream=None, window=None, alibi_slopes=None,
        n_splits: int | None = None, split_workspace: torch.Tensor | None = None,
        seqlens_k: torch.Tensor | None = None):
    """Forward attention. q [B,Hq,Sq,D], k/v [B,Hkv,Sk,D] bf16 CUDA.

    ``window=(left, right)``, ``alibi_slopes`` (fp32 [Hq]) and ``seqlens_k``
    (int32 [B] key counts: the key padding mask) select the score modification
    of fa_fwd_mod (include/fa.h); a row that sees no key gets O = 0, LSE = -inf.  ``n_splits`` (0: automatic)
    runs the split-KV form fa_fwd_split; its workspace is ``split_workspace``
    (uint8 CUDA) or allocated here.
    Returns (o [B,Hq,Sq,D] bf16, lse [B,Hq,Sq] fp32, natural log).
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n)
    B, Hq, Sq, D = q.shape
    _, Hkv, Sk, _ = k.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _new(q.shape, q.dtype, q.device, stream)
    if lse is None:
        lse = _new((B, Hq, Sq), torch.float32, q.device, stream)
    mod = _score_mod(causal, window, alibi_slopes, Hq, seqlens_k, B)
    if n_splits is not None:
        if mod is None and causal:
            mod = ScoreMod(-1, 0, None, None)
        ws_bytes = fwd_split_workspace_bytes(B, Hq, Sq, Sk, D, n_splits)
        if split_workspace is None:
            split_workspace = _new((max(ws_bytes, 1),), torch.uint8, q.device, stream,
                                   returned=False)
        rc = lib().fa_fwd_split(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, Sq,
                                Sk, D, None if mod is None else ctypes.byref(mod), float(scale),
                                int(n_splits), _ptr(split_workspace),
                                split_workspace.numel() * split_workspace.element_size(),
                                _stream(stream))
        if rc != FA_OK:
            raise FAError("fa_fwd_split", rc)
        return out, lse
    if mod is None:
        rc = lib().fa_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, Sq, Sk, D,
                          int(bool(causal)), float(scale), _stream(stream))
    else:
        rc = lib().fa_fwd_mod(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, Hq, Hkv, Sq,
                              Sk, D, ctypes.byref(mod), float(scale), _stream(stream))
    if rc != FA_OK:
        raise FAError("fa_fwd_mod" if mod is not None else "fa_fwd", rc)
    return out, lse


def fwd_split_count(B, Hq, Sq, Sk, sm_count: int = 0) -> int:
    """Splits fa_fwd_split uses for n_splits = 0 (sm_count 0: current device)."""
    return int(lib().fa_fwd_split_count(B, Hq, Sq, Sk, int(sm_count)))


def fwd_split_workspace_bytes(B, Hq, Sq, Sk, D, n_splits: int = 0) -> int:
    return int(lib().fa_fwd_split_workspace_bytes(B, Hq, Sq, Sk, D, int(n_splits)))


def lse_merge(o_parts: torch.Tensor, lse_parts: torch.Tensor, out: torch.Tensor | None = None,
              lse: torch.Tensor | None = None, stream=None):
    """Log-sum-exp merge of parts over disjoint key sets (fa_lse_merge).

    o_parts [n, ..., D] fp32 and lse_parts [n, ...] fp32 (natural log, -inf for
    an empty part), contiguous CUDA.  Returns (o [..., D] bf16, lse [...] fp32).
    """
    for t, n in ((o_parts, "o_parts"), (lse_parts, "lse_parts")):
        if not t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous():
            raise TypeError(f"{n} must be a contiguous fp32 CUDA tensor")
    if tuple(lse_parts.shape) != tuple(o_parts.shape[:-1]):
        raise ValueError("lse_parts must be o_parts' shape without the last dimension")
    n, D = o_parts.shape[0], o_parts.shape[-1]
    rows = lse_parts[0].numel() if n > 0 else 0
    if out is None:
        out = _new(o_parts.shape[1:], torch.bfloat16, o_parts.device, stream)
    if lse is None:
        lse = _new(lse_parts.shape[1:], torch.float32, o_parts.device, stream)
    rc = lib().fa_lse_merge(_ptr(o_parts), _ptr(lse_parts), int(n), _ptr(out), _ptr(lse),
                            int(rows), int(D), _stream(stream))
    if rc != FA_OK:
        raise FAError("fa_lse_merge", rc)
    return out, lse


def bwd_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, deterministic=False) -> int:
    return int(lib().fa_bwd_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, int(bool(deterministic))))


def bwd(q, k, v, o, do, lse, causal: bool = False, scale: float | None = None,
        deterministic: bool = False, workspace: torch.Tensor | None = None,
        dq=None, dk=None, dv=None, stream=None, window=None, alibi_slopes=None,
        seqlens_k=None):
    """Backward attention. Returns (dq, dk, dv) bf16, same shapes as q, k, v.
    ``window`` / ``alibi_slopes`` / ``seqlens_k`` as in fwd (must match the
    forward call)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (do, "do")):
        _check(t, n)
    if lse.dtype != torch.float32 or not lse.is_cuda or not lse.is_contiguous():
        raise TypeError("lse must be a contiguous fp32 CUDA tensor")
    B, Hq, Sq, D = q.shape
    _, Hkv, Sk, _ = k.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    need = bwd_workspace_bytes(B, Hq, Hkv, Sq, Sk, D, deterministic)
    if workspace is None:
        workspace = _new((need,), torch.uint8, q.device, stream, returned=False)
    dq, dk, dv = (_new(x.shape, x.dtype, x.device, stream) if g is None else g
                  for x, g in ((q, dq), (k, dk), (v, dv)))
    mod = _score_mod(causal, window, alibi_slopes, Hq, seqlens_k, B)
    if mod is None:
        rc = lib().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                          _ptr(dk), _ptr(dv), B, Hq, Hkv, Sq, Sk, D, int(bool(causal)),
                          float(scale), _ptr(workspace), workspace.numel(),
                          int(bool(deterministic)), _stream(stream))
    else:
        rc = lib().fa_bwd_mod(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                              _ptr(dk), _ptr(dv), B, Hq, Hkv, Sq, Sk, D, ctypes.byref(mod),
                              float(scale), _ptr(workspace), workspace.numel(),
                              int(bool(deterministic)), _stream(stream))
    if rc != FA_OK:
        raise FAError("fa_bwd_mod" if mod is not None else "fa_bwd", rc)
    return dq, dk, dv


def fwd_status(stream=None) -> int:
    """Synchronise and return (then clear) the forward kernels' timeout record."""
    return int(lib().fa_fwd_status(_stream(stream)))


def bwd_status(workspace: torch.Tensor, stream=None) -> int:
    return int(lib().fa_bwd_status(_ptr(workspace), _stream(stream)))


def exp2_test(x: torch.Tensor, which: int, stream=None) -> torch.Tensor:
    """2^x through the kernel's MUFU path (which=0), polynomial path (which=1) or
    packed two-lane polynomial path (which=2)."""
    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise TypeError("x must be a contiguous fp32 CUDA tensor")
    y = _new(x.shape, x.dtype, x.device, stream)
    rc = lib().fa_exp2_test(_ptr(x), _ptr(y), x.numel(), int(which), _stream(stream))
    if rc != FA_OK:
        raise FAError("fa_exp2_test", rc)
    return y


def wait_test(which: int, flag: torch.Tensor | None = None, stream=None) -> int:
    """Run one of the kernels' bounded waits (fa_wait_test); returns the status it
    wrote: FA_OK or FA_ERR_TIMEOUT (6).  flag: an int32 CUDA scalar for which=0."""
    device = flag.device if flag is not None else torch.device("cuda", torch.cuda.current_device())
    status = _new((1,), torch.int32, device, stream)
    with torch.cuda.stream(stream):  # (None: the current one)
        status.fill_(-1)
    rc = lib().fa_wait_test(None if flag is None else _ptr(flag), int(which), _ptr(status),
                            _stream(stream))
    if rc != FA_OK:
        raise FAError("fa_wait_test", rc)
    with torch.cuda.stream(stream):
        return int(status.item())


def last_launch_count() -> int:
    return int(lib().fa_last_launch_count())


def set_timing_events(start: "torch.cuda.Event | None", stop: "torch.cuda.Event | None") -> None:
    """Record ``start``/``stop`` around the main kernel of the next fwd/bwd call
    made by this thread (events must be created with timing enabled)."""
    for e in (start, stop):
        if e is not None and e.cuda_event == 0:
            e.record()  # torch creates the CUDA event lazily, on its first record
    ps = ctypes.c_void_p(start.cuda_event) if start is not None else None
    pe = ctypes.c_void_p(stop.cuda_event) if stop is not None else None
    rc = lib().fa_set_timing_events(ps, pe)
    if rc != FA_OK:
        raise FAError("fa_set_timing_events", rc)


BWD_KERNEL_AUTO, BWD_KERNEL_ONE_SM, BWD_KERNEL_PAIR = 0, 1, 2


def set_bwd_kernel(kind: int) -> int:
    """Backward main kernel for head dim 128, atomic dQ, no score modification
    (fa_set_bwd_kernel): BWD_KERNEL_AUTO, BWD_KERNEL_ONE_SM or BWD_KERNEL_PAIR
    (CTA pairs, 2-CTA MMA).  Returns the previous setting."""
    prev = ctypes.c_int(0)
    rc = lib().fa_set_bwd_kernel(int(kind), ctypes.byref(prev))
    if rc != FA_OK:
        raise FAError("fa_set_bwd_kernel", rc)
    return prev.value


class _Attention(torch.autograd.Function):
    """fwd in forward (saving O and LSE), bwd in backward; nothing else runs."""

    @staticmethod
    def forward(ctx, q, k, v, causal, scale, window, alibi_slopes, deterministic, seqlens_k):
        o, lse = fwd(q, k, v, causal=causal, scale=scale, window=window,
                     alibi_slopes=alibi_slopes, seqlens_k=seqlens_k)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.args = (causal, scale, window, alibi_slopes, deterministic, seqlens_k)
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse = ctx.saved_tensors
        causal, scale, window, alibi_slopes, deterministic, seqlens_k = ctx.args
        dq, dk, dv = bwd(q, k, v, o, do.contiguous(), lse, causal=causal, scale=scale,
                         deterministic=deterministic, window=window, alibi_slopes=alibi_slopes,
                         seqlens_k=seqlens_k)
        return dq, dk, dv, None, None, None, None, None, None


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
              scale: float | None = None, window=None, alibi_slopes=None,
              deterministic: bool = False, seqlens_k=None) -> torch.Tensor:
    """Exact attention as a differentiable op: O = softmax(scale q k^T + mods) v.

    q [B,Hq,Sq,D], k/v [B,Hkv,Sk,D] bf16 CUDA; ``causal``, ``window``,
    ``alibi_slopes`` and ``seqlens_k`` as in fwd; ``deterministic`` selects the
    backward mode.  O.backward() runs fa_bwd (the slopes get no gradient, and the
    gradients cannot be differentiated again: RuntimeError).  Returns O bf16.
    """
    return _Attention.apply(q, k, v, causal, scale, window, alibi_slopes, deterministic,
                            seqlens_k)


# The calls below also serve single tokens, where the host's time is most of a
# call's, so their checks and allocations are compiled (csrc/binding.cpp).  With
# ``stream`` a call runs there and what it allocates is that stream's; the caller
# orders it behind the arguments' last writers, and the results' readers behind it.

_COMPILED = None


def _compiled():
    global _COMPILED
    if _COMPILED is None:
        lib()  # raises if the library has not been built
        from . import _binding
        _binding.set_error(FAError)
        _COMPILED = _binding
    return _COMPILED


def _var_window(causal, window):
    if window is None:
        return -1, (0 if causal else -1)
    if causal:
        raise ValueError("give the causal mask as window=(-1, 0), not with causal=True")
    return int(window[0]), int(window[1])


def _left(window_left):
    """A window's left side for the C ABI: -1 for none; a C int would not hold the largest."""
    return -1 if window_left is None else max(-1, min(int(window_left), 2 ** 31 - 1))


def varlen_workspace_bytes(B, T, Hq, Hkv, D, backward=False, deterministic=False, window=None,
                           sinks: int = 0) -> int:
    """Workspace bytes of fwd_varlen or bwd_varlen; a backward with ``sinks`` takes more, by
    its ``window``."""
    return int(lib().fa_varlen_sink_workspace_bytes(
        B, T, Hq, Hkv, D, int(bool(backward)), int(bool(deterministic)),
        _left(_var_window(False, window)[0]), int(sinks)))


def fwd_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
               causal: bool = False, scale: float | None = None, window=None,
               out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, stream=None, sinks: int = 0):
    """Forward attention over packed sequences (fa_fwd_varlen, fa_fwd_varlen_sink).

    q [T,Hq,D], k/v [T,Hkv,D] bf16 CUDA, elements contiguous, tokens and heads at
    any stride that is a multiple of 8 (slices of a fused projection);
    ``cu_seqlens`` int32 [B+1]: sequence b is tokens cu_seqlens[b] ..
    cu_seqlens[b+1]-1.  ``causal`` / ``window`` as in fwd, inside each sequence;
    the first ``sinks`` tokens (at most 128) stay visible behind the window's left side.
    Returns (o [T,Hq,D] bf16, lse [Hq,T] fp32); tokens of no sequence are not
    written.  fwd_status() reports a cu_seqlens that does not ascend in [0, T].
    """
    wl, wr = _var_window(causal, window)
    return _compiled().fwd_varlen(q, k, v, cu_seqlens, wl, wr, scale, out, lse, workspace, stream,
                                  sinks)


def bwd_varlen(q, k, v, o, do, lse, cu_seqlens, causal: bool = False, scale: float | None = None,
               window=None, deterministic: bool = False, workspace: torch.Tensor | None = None,
               dq=None, dk=None, dv=None, stream=None, sinks: int = 0):
    """Backward of fwd_varlen (fa_bwd_varlen, fa_bwd_varlen_sink).  Returns (dq [T,Hq,D], dk, dv
    [T,Hkv,D]) bf16, contiguous; tokens of no sequence are not written.  o, do
    and lse are contiguous; the other arguments as in fwd_varlen, and as given
    to it."""
    wl, wr = _var_window(causal, window)
    return _compiled().bwd_varlen(q, k, v, o, do, lse, cu_seqlens, wl, wr, scale, deterministic,
                                  workspace, dq, dk, dv, stream, sinks)


class _AttentionVarlen(torch.autograd.Function):
    """fwd_varlen in forward (saving O and LSE), bwd_varlen in backward."""

    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, causal, scale, window, deterministic, sinks):
        # tokens of no sequence: zeros, so that neither O nor a gradient holds
        # uninitialised memory
        o = torch.zeros(q.shape, dtype=q.dtype, device=q.device)
        _, lse = fwd_varlen(q, k, v, cu_seqlens, causal=causal, scale=scale, window=window, out=o,
                            sinks=sinks)
        ctx.save_for_backward(q, k, v, o, lse, cu_seqlens)
        ctx.args = (causal, scale, window, deterministic, sinks)
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, cu_seqlens = ctx.saved_tensors
        causal, scale, window, deterministic, sinks = ctx.args
        grads = [torch.zeros(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v)]
        bwd_varlen(q, k, v, o, do.contiguous(), lse, cu_seqlens, causal=causal, scale=scale,
                   window=window, deterministic=deterministic, dq=grads[0], dk=grads[1],
                   dv=grads[2], sinks=sinks)
        return (*grads, None, None, None, None, None, None)


def attention_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                     causal: bool = False, scale: float | None = None, window=None,
                     deterministic: bool = False, sinks: int = 0) -> torch.Tensor:
    """attention() over packed sequences: q [T,Hq,D], k/v [T,Hkv,D] bf16 CUDA,
    ``cu_seqlens`` int32 [B+1], ``sinks`` (see fwd_varlen).  Tokens of no sequence get zeros
    in O and in every gradient.  A training step can be captured into a CUDA graph
    after a step on a side stream; no other graph of the same leaves may be alive
    then.  The gradients cannot be differentiated again (RuntimeError).  Returns O
    [T,Hq,D] bf16."""
    return _AttentionVarlen.apply(q, k, v, cu_seqlens, causal, scale, window, deterministic, sinks)


def rope_table(positions: int, rot: int, base: float = 10000.0, device="cuda", stream=None):
    """cos and sin fp32 [positions, rot/2] of the angles p base^(-2i/rot), taken in 64 bits
    (fa_rope_table)."""
    device = torch.device(device)
    if device.type != "cuda":
        raise TypeError("rope_table fills CUDA tensors")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(device):
        cos, sin = (_new((max(positions, 0), max(rot, 0) // 2), torch.float32, device, stream)
                    for _ in range(2))
        rc = lib().fa_rope_table(_ptr(cos), _ptr(sin), int(positions), int(rot), float(base),
                                 _stream(stream))
    if rc != FA_OK:
        raise FAError("fa_rope_table", rc)
    return cos, sin


def norm_rope_fwd(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor, k_weight: torch.Tensor,
                  cos: torch.Tensor, sin: torch.Tensor, positions: torch.Tensor, eps: float = 1e-6,
                  interleaved: bool = False, q_out=None, k_out=None, zero_skipped: bool = False,
                  stream=None):
    """RMS norms of query and key heads and their rotation by position (fa_norm_rope_fwd).

    q [T,Hq,D], k [T,Hkv,D] bf16 CUDA, elements contiguous, tokens and heads at any stride
    that is a multiple of 8 (slices of a fused projection); weights [D], fp32 or bf16;
    ``cos``, ``sin`` fp32 [P,rot/2] (rope_table): the first ``rot`` elements of a head are
    rotated, in pairs (i, i + rot/2), or (2i, 2i + 1) with ``interleaved``; ``positions``
    int32 [T].  A token with a negative position is of no sequence: its rows are not
    written, or become zeros with ``zero_skipped``.  fwd_status() reports positions from P on,
    which count as such.  ``q_out``, ``k_out``: like q and k, of any such strides, also q
    and k themselves.  Returns (q_out, k_out) bf16.
    """
    return _compiled().norm_rope_fwd(q, k, q_weight, k_weight, cos, sin, positions, float(eps),
                                     interleaved, q_out, k_out, zero_skipped, stream)


def norm_rope_workspace_bytes(T, Hq, Hkv, D) -> int:
    """Workspace bytes of norm_rope_bwd on the current device."""
    return int(lib().fa_norm_rope_workspace_bytes(T, Hq, Hkv, D))


def norm_rope_bwd(q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, eps: float = 1e-6,
                  interleaved: bool = False, dq=None, dk=None, dq_weight=None, dk_weight=None,
                  workspace: torch.Tensor | None = None, zero_skipped: bool = False, stream=None):
    """Backward of norm_rope_fwd (fa_norm_rope_bwd), whose arguments it takes as given there.
    Returns (dq, dk bf16, dq_weight, dk_weight fp32 [D]); the same bits in every run."""
    return _compiled().norm_rope_bwd(q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out,
                                     float(eps), interleaved, dq, dk, dq_weight, dk_weight,
                                     workspace, zero_skipped, stream)


class _NormRope(torch.autograd.Function):
    """norm_rope_fwd in forward, norm_rope_bwd in backward; nothing else runs."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved):
        ctx.save_for_backward(q, k, q_weight, k_weight, cos, sin, positions)
        ctx.args = (eps, interleaved)
        return norm_rope_fwd(q, k, q_weight, k_weight, cos, sin, positions, eps=eps,
                             interleaved=interleaved, zero_skipped=True)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq_out, dk_out):
        q, k, q_weight, k_weight, cos, sin, positions = ctx.saved_tensors
        eps, interleaved = ctx.args
        dq, dk, dqw, dkw = norm_rope_bwd(q, k, q_weight, k_weight, cos, sin, positions,
                                         dq_out.contiguous(), dk_out.contiguous(), eps=eps,
                                         interleaved=interleaved, zero_skipped=True)
        return dq, dk, dqw.to(q_weight.dtype), dkw.to(k_weight.dtype), None, None, None, None, None


def norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor, k_weight: torch.Tensor,
              cos: torch.Tensor, sin: torch.Tensor, positions: torch.Tensor, eps: float = 1e-6,
              interleaved: bool = False):
    """norm_rope_fwd as a differentiable op: gradients for q, k and the weights (those in the
    weights' type).  Tokens with a negative position get zeros in the results and in every
    gradient.  A training step can be captured into a CUDA graph, as with attention_varlen.
    The gradients cannot be differentiated again (RuntimeError).  Returns (q, k) bf16,
    contiguous."""
    return _NormRope.apply(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved)


def cache4_empty(num_pages: int, Hkv: int, D: int, page_size: int = 64, device="cuda"):
    """A paged 4-bit key/value cache (include/fa.h, fa_cache4_page_bytes): uint8
    [num_pages, Hkv, bytes of a page and head], zeroed.  page_size: 16, 32, 64 or
    128 tokens.  The bytes are opaque; cache4_read returns the values."""
    nbytes = int(lib().fa_cache4_page_bytes(Hkv, D, page_size))
    if nbytes == 0:
        raise FAError("fa_cache4_page_bytes", 2)
    return torch.zeros((num_pages, Hkv, nbytes // Hkv), dtype=torch.uint8, device=device)


def cache4_append(cache: torch.Tensor, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor,
                  cache_lens: torch.Tensor, cu_seqlens: torch.Tensor | None = None, stream=None):
    """Quantises and stores new tokens (fa_cache4_append).

    k, v [T,Hkv,D] bf16 CUDA, elements contiguous; ``page_table`` int32 [B,width];
    ``cache_lens`` int32 [B]: tokens held before, which is where the new ones go;
    ``cu_seqlens`` int32 [B+1] packs several per sequence, None means one each
    (T == B).  cache_lens is left as it is: add the new tokens to it afterwards.
    """
    _compiled().cache4_append(cache, k, v, page_table, cache_lens, cu_seqlens, stream)


def cache4_append_slots(cache: torch.Tensor, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                        stream=None):
    """Quantises and stores new tokens by slot (fa_cache4_append_slots): row i of k, v
    [T,Hkv,D] goes to slot ``slots[i]`` (int64 [T], as page_update returns them), a negative
    one nowhere."""
    _compiled().cache4_append_slots(cache, k, v, slots, stream)


def page_pool(num_pages: int, device="cuda"):
    """A pool of free pages 0 .. num_pages - 1 for page_update: (free_pages int32
    [num_pages], a stack, and free_count int32 [1])."""
    return (torch.arange(num_pages, dtype=torch.int32, device=device),
            torch.full((1,), num_pages, dtype=torch.int32, device=device))


def page_update(page_table: torch.Tensor, free_pages: torch.Tensor, free_count: torch.Tensor,
                lens: torch.Tensor, new_lens: torch.Tensor, page_size: int, T: int,
                window_left: int | None = None, sinks: int = 0, cu_seqlens=None, positions=None,
                slots=None, stream=None):
    """Page tables for the lengths to come (fa_page_update), in place.

    ``page_table`` int32 [B,width]; ``free_pages``, ``free_count``: the pool (page_pool);
    ``lens``, ``new_lens`` int32 [B]: tokens held and to be held.  Entries past the new
    length, and those that a window of ``window_left`` tokens with ``sinks`` hides from the
    last token's query on, give their pages back; entries for new tokens take pages.  A
    page belongs to one entry: tables that share pages are not for this call.  A table
    begins as -1 everywhere.
    Returns (cu_seqlens int32 [B+1], positions int32 [T], slots int64 [T]) of the new
    tokens, packed in order; ``T`` is the rows they have, and rows past the last get -1.
    cache4_status() reports a pool or T that was too small, and lengths past the table.
    """
    return _compiled().page_update(page_table, free_pages, free_count, lens, new_lens, page_size, T,
                                   _left(window_left), sinks, cu_seqlens, positions, slots, stream)


def cache4_read(cache: torch.Tensor, page_table: torch.Tensor, first: torch.Tensor | None,
                count: torch.Tensor, S: int, D: int, k=None, v=None, stream=None):
    """The values the cache holds (fa_cache4_read): slots first[b] .. first[b] +
    count[b] - 1 of every sequence (``first`` None: from 0) as bf16 k, v
    [B,Hkv,S,D], zero from count[b] on."""
    return _compiled().cache4_read(cache, page_table, first, count, S, D, k, v, stream)


def cache4_attend_workspace_bytes(B, Hq, Hkv, D, weight_slots: int = 0) -> int:
    """Workspace bytes of cache4_attend on the current device; weight_slots: the last
    dimension of its weights, 0 without."""
    return int(lib().fa_cache4_attend_workspace_bytes(B, Hq, Hkv, D, int(weight_slots)))


def cache4_attend(q: torch.Tensor, cache: torch.Tensor, page_table: torch.Tensor,
                  cache_lens: torch.Tensor, scale: float | None = None,
                  weights: torch.Tensor | None = None, weights_out: torch.Tensor | None = None,
                  out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream=None,
                  window_left: int | None = None, sinks: int = 0):
    """One query token per sequence attends to its cache (fa_cache4_attend,
    fa_cache4_attend_sink).

    q [B,Hq,D] bf16 CUDA, elements contiguous; ``cache_lens`` int32 [B].
    ``weights`` fp32 [B,Hkv,slots] has the tokens' softmax weights, summed over each
    kv head's query heads, added to it in place, or to a copy in ``weights_out``;
    ``weights_out`` alone gets this step's.  Tokens that an append adds later start
    at what the tensor holds there, so it begins as zeros.  ``slots`` is at least
    every length: tokens behind it are left out of all results and cache4_status()
    reports them.
    ``window_left``: the query, which is the last token's, sees the ``window_left`` tokens
    before it and the first ``sinks``; the pages of the others are not looked up.
    Returns (o [B,Hq,D] bf16, lse [B,Hq] fp32); o = 0, lse = -inf without tokens.
    """
    return _compiled().cache4_attend(q, cache, page_table, cache_lens, scale, weights, weights_out,
                                     out, lse, workspace, stream, _left(window_left), sinks)


def cache4_evict(cache: torch.Tensor, page_table: torch.Tensor, cache_lens: torch.Tensor,
                 weights: torch.Tensor, out_page_table: torch.Tensor, D: int, budget: int,
                 recent: int = 0, src=None, weights_out=None, lens_out=None, stream=None):
    """Keeps at most ``budget`` tokens per (sequence, kv head): the latest ``recent``
    and the largest ``weights`` [B,Hkv,slots] of the others, copied in order to the
    pages of ``out_page_table`` (fa_cache4_evict), which no table in use may name.

    Returns (src int32 [B,Hkv,budget]: each kept token's old slot, -1 behind the
    last; weights fp32 [B,Hkv,budget], 0 behind the last; lens int32 [B]).
    For the next steps' cache4_attend copy the weights into a tensor with slots for
    the tokens to come, zeros there.
    """
    return _compiled().cache4_evict(cache, page_table, cache_lens, weights, out_page_table, D, budget,
                                    recent, src, weights_out, lens_out, stream)


def cache4_status(stream=None) -> int:
    """Synchronise and return (then clear) what the cache calls recorded: a page id
    or length out of range (1), a device-side wait that ran out (6)."""
    return int(lib().fa_cache4_status(_stream(stream)))
