"""ctypes binding of libattn_sink.so (argument marshalling only).

Every step of the computation runs in the library's CUDA kernels; this module
only checks tensor dtypes/devices, allocates outputs with torch and passes raw
pointers, sizes and the current CUDA stream through the C ABI.  There is no
fallback: if the shared library is missing the import fails loudly.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libattn_sink.so")

OK, ERR_INVALID, ERR_UNSUPPORTED, ERR_CUDA, ERR_DEVICE = 0, -1, -2, -3, -4
DEV_PAGE_OOB, DEV_SEQLEN_OOB, DEV_TIMEOUT, DEV_LAYOUT = 1, 2, 4, 8
DEV_ORDER, DEV_TREE = 16, 32
DEV_VALUE, DEV_PROB, DEV_POOL = 64, 128, 256

_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_longlong
_F = ctypes.c_float

_SIGS = {
    "attn_sink_fwd": [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P,
                      _P],
    "attn_sink_decode_paged": [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _P, _I, _I, _F, _P, _P, _P],
    "attn_sink_decode_paged_noalloc": [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _P, _I, _I, _F, _P,
                                       _P, _P],
    "attn_sink_bwd": [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                      _I, _F, _P, _P, _P, _P, _P],
    "attn_sink_fwd_host": [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P],
    "attn_sink_fwd_strided": [_P, _P, _P, _L, _L, _L, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                              _I, _F, _P, _P, _P],
    "attn_sink_bwd_strided": [_P, _P, _P, _L, _L, _L, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I,
                              _I, _I, _I, _I, _F, _P, _P, _P, _L, _L, _L, _P, _P],
    "attn_sink_kv_append": [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P],
    "attn_sink_decode_paged_append": [_P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _P, _I, _I, _F,
                                      _P, _P, _P],
    "attn_sink_fwd_paged": [_P, _P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _I,
                            _I, _I, _F, _P, _P, _P],
    "attn_sink_rope": [_P, _P, _P, _P, _L, _L, _L, _L, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P],
    "attn_sink_rope_kv_append": [_P, _P, _P, _P, _L, _L, _L, _L, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I,
                                 _I, _I, _I, _I, _F, _P, _P, _P],
    "attn_sink_tree_paged": [_P, _P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _I, _I, _F,
                             _P, _P, _P],
    "attn_sink_kv_compact": [_P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P],
    "attn_sink_decode_paged_weights": [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _P, _I, _I, _F, _P, _I, _I,
                                       _P, _P, _P],
    "attn_sink_decode_paged_weights_bounded": [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _I, _P, _I, _I, _F,
                                               _P, _I, _I, _P, _P, _P],
    "attn_sink_evict_paged": [_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P],
    "attn_sink_visible_ranges": [_P, _I, _I, _I, _P, _P],
    "attn_sink_visible_slots": [_P, _P, _I, _I, _I, _I, _I, _I, _P, _I, _P],
    "attn_sink_device_status": [_P],
    "attn_sink_kv_append_q8": [_P, _P, _L, _L, _P, _P, _P] + [_I] * 10 + [_P] * 5,
    "attn_sink_decode_paged_q8": [_P] * 5 + [_I, _I, _P, _I, _P] + [_I] * 7 + [_P, _I, _I, _F, _P, _P, _P],
    "attn_sink_fwd_paged_q8": [_P] * 5 + [_I, _I, _P, _I, _P, _P] + [_I] * 9 + [_P, _I, _I, _I, _F, _P, _P, _P],
    "attn_sink_verify_draft": [_P, _P, _L, _L, _I] + [_P] * 6 + [_I] * 4 + [_P] * 4,
    "attn_sink_pages_copy": [_P, _P, _I, _I, _P, _P, _I, _P],
    "attn_sink_pages_fork": [_P] * 4 + [_I] * 5 + [_P] * 3,
    "attn_sink_pages_release": [_P] * 4 + [_I] * 4 + [_P],
    "attn_sink_pages_reserve": [_P, _P, _I] + [_P] * 4 + [_I] * 4 + [_P, _P],
    "attn_sink_pages_compact": [_P, _P, _I] + [_P] * 3 + [_I] * 4 + [_P, _P],
    "attn_sink_selftest_wait": [_I, _P],
    "attn_sink_last_error": [],
    "attn_sink_version": [],
}

EXPORTS = tuple(_SIGS)


class AttnSinkError(RuntimeError):
    def __init__(self, fn, code, msg):
        super().__init__(f"{fn} returned {code}: {msg}")
        self.code = code


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it first (python -m paged_kv_sink_gb300.build)")
    lib = ctypes.CDLL(path)
    for name, args in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_char_p if name in ("attn_sink_last_error", "attn_sink_version") else ctypes.c_int
    return lib


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        _lib = load()
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _made(stream, make, *args, **kw):
    """An output that a call allocates.  It belongs to the stream that the call launches on
    (None: the current one), so that its memory is not handed on while a kernel there
    still writes it, even when the caller drops it at once, and it is recorded on the current
    stream, where the caller goes on with it."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        t = make(*args, **kw)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _check(name, rc):
    if rc != OK:
        msg = lib().attn_sink_last_error().decode()
        raise AttnSinkError(name, rc, msg)


def _need(t, dtype, name, dev=True):
    if t is None:
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dev and not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise TypeError(f"{name} must be contiguous")


def attn_sink_fwd(q, k, v, sink, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k,
                  win_first=0, win_last=0, causal=True, scale=0.0, out=None, lse=None,
                  return_lse=True, stream=None):
    """Varlen forward with a sink.  q (Tq,Hq,d), k/v (Tk,Hkv,d) bf16 CUDA; returns (out, lse)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, n)
    _need(sink, torch.float32, "sink")
    _need(cu_seqlens_q, torch.int32, "cu_seqlens_q")
    _need(cu_seqlens_k, torch.int32, "cu_seqlens_k")
    tq, hq, d = q.shape
    hkv = k.shape[1]
    if out is None:
        out = _made(stream, torch.empty_like, q)
    if lse is None and return_lse:
        lse = _made(stream, torch.empty, (hq, tq), dtype=torch.float32, device=q.device)
    rc = lib().attn_sink_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(sink), _ptr(cu_seqlens_q),
                             _ptr(cu_seqlens_k), cu_seqlens_q.numel() - 1, tq, k.shape[0], hq, hkv,
                             d, int(max_seqlen_q), int(max_seqlen_k), int(win_first), int(win_last),
                             1 if causal else 0, float(scale), _ptr(out), _ptr(lse), _stream(stream))
    _check("attn_sink_fwd", rc)
    return out, lse


def attn_sink_fwd_host(q, k, v, sink, cu_seqlens_q, cu_seqlens_k, win_first=0, win_last=0, causal=True,
                       scale=0.0, out=None, lse=None, return_lse=True, stream=None):
    """attn_sink_fwd on host (CPU, preferably pinned) tensors: the library moves
    each request's rows to the device and back, pipelined against the kernels.
    Returns (out, lse) as host tensors; they are valid after ``stream`` (default:
    the current CUDA stream) is synchronised."""
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _need(t, torch.bfloat16, n, dev=False)
    _need(sink, torch.float32, "sink", dev=False)
    _need(cu_seqlens_q, torch.int32, "cu_seqlens_q", dev=False)
    _need(cu_seqlens_k, torch.int32, "cu_seqlens_k", dev=False)
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (sink, "sink"), (cu_seqlens_q, "cu_seqlens_q"),
                 (cu_seqlens_k, "cu_seqlens_k")):
        if t is not None and t.is_cuda:
            raise TypeError(f"{n} must be a host tensor")
    tq, hq, d = q.shape
    hkv = k.shape[1]
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, pin_memory=True)
    if lse is None and return_lse:
        lse = torch.empty((hq, tq), dtype=torch.float32, pin_memory=True)
    rc = lib().attn_sink_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(sink), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k),
                                  cu_seqlens_q.numel() - 1, hq, hkv, d, int(win_first), int(win_last),
                                  1 if causal else 0, float(scale), _ptr(out), _ptr(lse), _stream(stream))
    _check("attn_sink_fwd_host", rc)
    return out, lse


def attn_sink_decode_paged(q, k_cache, v_cache, page_table, seqlens, sink=None, win_first=0,
                           win_last=0, scale=0.0, out=None, lse=None, return_lse=True, stream=None,
                           _entry="attn_sink_decode_paged"):
    """Paged decode.  q (B,Hq,d); caches (P,ps,Hkv,d); page_table (B,maxp) int32; seqlens (B,)."""
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, torch.bfloat16, n)
    _need(page_table, torch.int32, "page_table")
    _need(seqlens, torch.int32, "seqlens")
    _need(sink, torch.float32, "sink")
    B, hq, d = q.shape
    npages, ps, hkv, _ = k_cache.shape
    if out is None:
        out = _made(stream, torch.empty_like, q)
    if lse is None and return_lse:
        lse = _made(stream, torch.empty, (B, hq), dtype=torch.float32, device=q.device)
    rc = getattr(lib(), _entry)(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
                                page_table.shape[1], _ptr(seqlens), B, hq, hkv, d, ps, npages,
                                _ptr(sink), int(win_first), int(win_last), float(scale),
                                _ptr(out), _ptr(lse), _stream(stream))
    _check(_entry, rc)
    return out, lse


def attn_sink_decode_paged_noalloc(q, k_cache, v_cache, page_table, seqlens, sink=None, win_first=0,
                                   win_last=0, scale=0.0, out=None, lse=None, return_lse=True,
                                   stream=None):
    """Allocation-free paged decode: the library allocates no device memory
    for the call (its scratch is a static device array).  Outputs are still
    allocated here by torch unless ``out``/``lse`` are given."""
    return attn_sink_decode_paged(q, k_cache, v_cache, page_table, seqlens, sink, win_first, win_last,
                                  scale, out, lse, return_lse, stream,
                                  _entry="attn_sink_decode_paged_noalloc")


def _row_view(base, col0, heads, d):
    """(pointer, row stride) of columns [col0, col0 + heads) of a (T, C, d) buffer."""
    if base.dim() != 3 or base.stride(2) != 1 or base.stride(1) != d:
        raise TypeError("packed buffer must be (T, C, d) with contiguous rows")
    return ctypes.c_void_p(base.data_ptr() + col0 * d * base.element_size()), base.stride(0)


def attn_sink_fwd_qkvpacked(qkv, hkv, sink, cu_seqlens_q, max_seqlen_q, win_first=0, win_last=0,
                            causal=True, scale=0.0, out=None, lse=None, return_lse=True, stream=None):
    """Self-attention forward on a packed (T, hq + 2*hkv, d) QKV buffer (a
    (T, 3, H, d) buffer is the same with hkv = H after a view).  Returns (out, lse)."""
    if qkv.dim() == 4:
        qkv = qkv.reshape(qkv.shape[0], -1, qkv.shape[-1])
    _need(qkv, torch.bfloat16, "qkv")
    _need(sink, torch.float32, "sink")
    _need(cu_seqlens_q, torch.int32, "cu_seqlens_q")
    T, C, d = qkv.shape
    hq = C - 2 * hkv
    qp, rs = _row_view(qkv, 0, hq, d)
    kp, _ = _row_view(qkv, hq, hkv, d)
    vp, _ = _row_view(qkv, hq + hkv, hkv, d)
    if out is None:
        out = _made(stream, torch.empty, (T, hq, d), dtype=qkv.dtype, device=qkv.device)
    if lse is None and return_lse:
        lse = _made(stream, torch.empty, (hq, T), dtype=torch.float32, device=qkv.device)
    rc = lib().attn_sink_fwd_strided(qp, kp, vp, rs, rs, rs, _ptr(sink), _ptr(cu_seqlens_q), _ptr(cu_seqlens_q),
                                     cu_seqlens_q.numel() - 1, T, T, hq, hkv, d, int(max_seqlen_q),
                                     int(max_seqlen_q), int(win_first), int(win_last), 1 if causal else 0,
                                     float(scale), _ptr(out), _ptr(lse), _stream(stream))
    _check("attn_sink_fwd_strided", rc)
    return out, lse


def attn_sink_fwd_kvpacked(q, kv, sink, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, max_seqlen_k, win_first=0,
                           win_last=0, causal=True, scale=0.0, out=None, lse=None, return_lse=True,
                           stream=None):
    """Forward with a packed (Tk, 2, hkv, d) KV buffer.  Returns (out, lse)."""
    _need(q, torch.bfloat16, "q")
    _need(kv, torch.bfloat16, "kv")
    _need(sink, torch.float32, "sink")
    tq, hq, d = q.shape
    tk, _, hkv, _ = kv.shape
    kv3 = kv.reshape(tk, 2 * hkv, d)
    kp, rs = _row_view(kv3, 0, hkv, d)
    vp, _ = _row_view(kv3, hkv, hkv, d)
    if out is None:
        out = _made(stream, torch.empty_like, q)
    if lse is None and return_lse:
        lse = _made(stream, torch.empty, (hq, tq), dtype=torch.float32, device=q.device)
    rc = lib().attn_sink_fwd_strided(_ptr(q), kp, vp, 0, rs, rs, _ptr(sink), _ptr(cu_seqlens_q),
                                     _ptr(cu_seqlens_k), cu_seqlens_q.numel() - 1, tq, tk, hq, hkv, d,
                                     int(max_seqlen_q), int(max_seqlen_k), int(win_first), int(win_last),
                                     1 if causal else 0, float(scale), _ptr(out), _ptr(lse), _stream(stream))
    _check("attn_sink_fwd_strided", rc)
    return out, lse


def attn_sink_bwd_qkvpacked(qkv, hkv, sink, out, lse, dout, cu_seqlens_q, max_seqlen_q, win_first=0,
                            win_last=0, causal=True, scale=0.0, dqkv=None, dsink=None, stream=None):
    """Backward of attn_sink_fwd_qkvpacked; returns (dqkv, dsink or None), dqkv in
    the layout of qkv."""
    shape4 = qkv.shape if qkv.dim() == 4 else None
    if qkv.dim() == 4:
        qkv = qkv.reshape(qkv.shape[0], -1, qkv.shape[-1])
    for t, n in ((qkv, "qkv"), (out, "out"), (dout, "dout")):
        _need(t, torch.bfloat16, n)
    _need(sink, torch.float32, "sink")
    _need(lse, torch.float32, "lse")
    T, C, d = qkv.shape
    hq = C - 2 * hkv
    dqkv = _made(stream, torch.empty_like, qkv) if dqkv is None else dqkv.reshape(T, C, d)
    if sink is not None and dsink is None:
        dsink = _made(stream, torch.empty_like, sink)
    qp, rs = _row_view(qkv, 0, hq, d)
    kp, _ = _row_view(qkv, hq, hkv, d)
    vp, _ = _row_view(qkv, hq + hkv, hkv, d)
    dqp, drs = _row_view(dqkv, 0, hq, d)
    dkp, _ = _row_view(dqkv, hq, hkv, d)
    dvp, _ = _row_view(dqkv, hq + hkv, hkv, d)
    rc = lib().attn_sink_bwd_strided(qp, kp, vp, rs, rs, rs, _ptr(sink), _ptr(out), _ptr(lse), _ptr(dout),
                                     _ptr(cu_seqlens_q), _ptr(cu_seqlens_q), cu_seqlens_q.numel() - 1, T, T, hq,
                                     hkv, d, int(max_seqlen_q), int(max_seqlen_q), int(win_first),
                                     int(win_last), 1 if causal else 0, float(scale), dqp, dkp, dvp, drs, drs,
                                     drs, _ptr(dsink), _stream(stream))
    _check("attn_sink_bwd_strided", rc)
    return (dqkv.reshape(shape4) if shape4 is not None else dqkv), dsink


def attn_sink_bwd_kvpacked(q, kv, sink, out, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                           max_seqlen_k, win_first=0, win_last=0, causal=True, scale=0.0, dq=None, dkv=None,
                           dsink=None, stream=None):
    """Backward of attn_sink_fwd_kvpacked; returns (dq, dkv, dsink or None), dkv in
    the (Tk, 2, hkv, d) layout of kv.  Rows of dkv past every request's last key
    are not written (pass a zeroed ``dkv`` if kv has such rows)."""
    for t, n in ((q, "q"), (kv, "kv"), (out, "out"), (dout, "dout")):
        _need(t, torch.bfloat16, n)
    _need(sink, torch.float32, "sink")
    _need(lse, torch.float32, "lse")
    tq, hq, d = q.shape
    tk, _, hkv, _ = kv.shape
    dq = _made(stream, torch.empty_like, q) if dq is None else dq
    dkv = _made(stream, torch.empty_like, kv) if dkv is None else dkv
    _need(dkv, torch.bfloat16, "dkv")
    if sink is not None and dsink is None:
        dsink = _made(stream, torch.empty_like, sink)
    kp, rs = _row_view(kv.reshape(tk, 2 * hkv, d), 0, hkv, d)
    vp, _ = _row_view(kv.reshape(tk, 2 * hkv, d), hkv, hkv, d)
    dkp, drs = _row_view(dkv.reshape(tk, 2 * hkv, d), 0, hkv, d)
    dvp, _ = _row_view(dkv.reshape(tk, 2 * hkv, d), hkv, hkv, d)
    rc = lib().attn_sink_bwd_strided(_ptr(q), kp, vp, 0, rs, rs, _ptr(sink), _ptr(out), _ptr(lse), _ptr(dout),
                                     _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), cu_seqlens_q.numel() - 1, tq, tk, hq,
                                     hkv, d, int(max_seqlen_q), int(max_seqlen_k), int(win_first),
                                     int(win_last), 1 if causal else 0, float(scale), _ptr(dq), dkp, dvp, 0, drs,
                                     drs, _ptr(dsink), _stream(stream))
    _check("attn_sink_bwd_strided", rc)
    return dq, dkv, dsink


def attn_sink_kv_append(k_new, v_new, k_cache, v_cache, page_table, seqlens, cu_new=None,
                        max_new=None, stream=None):
    """Writes the new K/V rows into the paged caches in place (see the C header)."""
    for t, n in ((k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, torch.bfloat16, n)
    _need(page_table, torch.int32, "page_table")
    _need(seqlens, torch.int32, "seqlens")
    _need(cu_new, torch.int32, "cu_new")
    npages, ps, hkv, d = k_cache.shape
    B = seqlens.numel()
    if max_new is None:
        max_new = 1 if cu_new is None else int((cu_new[1:] - cu_new[:-1]).max()) if B else 0
    rc = lib().attn_sink_kv_append(_ptr(k_new), _ptr(v_new), _ptr(cu_new), _ptr(seqlens), _ptr(page_table),
                                   page_table.shape[1], B, hkv, d, ps, npages, int(max_new), _ptr(k_cache),
                                   _ptr(v_cache), _stream(stream))
    _check("attn_sink_kv_append", rc)
    return k_cache, v_cache


def attn_sink_decode_paged_append(q, k_new, v_new, k_cache, v_cache, page_table, seqlens, sink=None,
                                  win_first=0, win_last=0, scale=0.0, out=None, lse=None,
                                  return_lse=True, stream=None):
    """Paged decode with the new token's K/V (k_new, v_new: (B, Hkv, d)) written into
    the caches first, in the same call."""
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, torch.bfloat16, n)
    _need(page_table, torch.int32, "page_table")
    _need(seqlens, torch.int32, "seqlens")
    _need(sink, torch.float32, "sink")
    B, hq, d = q.shape
    npages, ps, hkv, _ = k_cache.shape
    if out is None:
        out = _made(stream, torch.empty_like, q)
    if lse is None and return_lse:
        lse = _made(stream, torch.empty, (B, hq), dtype=torch.float32, device=q.device)
    rc = lib().attn_sink_decode_paged_append(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                             _ptr(page_table), page_table.shape[1], _ptr(seqlens), B, hq, hkv, d,
                                             ps, npages, _ptr(sink), int(win_first), int(win_last), float(scale),
                                             _ptr(out), _ptr(lse), _stream(stream))
    _check("attn_sink_decode_paged_append", rc)
    return out, lse


def attn_sink_fwd_paged(q, k_cache, v_cache, page_table, cu_seqlens_q, seqlens_k, max_seqlen_q,
                        max_seqlen_k, sink=None, k_new=None, v_new=None, win_first=0, win_last=0,
                        causal=True, scale=0.0, out=None, lse=None, return_lse=True, stream=None):
    """Varlen extend against a paged K/V cache; with k_new/v_new the chunk's K/V
    are appended into the cache first.  Returns (out, lse)."""
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (k_new, "k_new"), (v_new, "v_new")):
        _need(t, torch.bfloat16, n)
    _need(page_table, torch.int32, "page_table")
    _need(cu_seqlens_q, torch.int32, "cu_seqlens_q")
    _need(seqlens_k, torch.int32, "seqlens_k")
    _need(sink, torch.float32, "sink")
    tq, hq, d = q.shape
    npages, ps, hkv, _ = k_cache.shape
    if out is None:
        out = _made(stream, torch.empty_like, q)
    if lse is None and return_lse:
        lse = _made(stream, torch.empty, (hq, tq), dtype=torch.float32, device=q.device)
    rc = lib().attn_sink_fwd_paged(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache),
                                   _ptr(page_table), page_table.shape[1], _ptr(cu_seqlens_q), _ptr(seqlens_k),
                                   cu_seqlens_q.numel() - 1, tq, hq, hkv, d, ps, npages, int(max_seqlen_q),
                                   int(max_seqlen_k), _ptr(sink), int(win_first), int(win_last),
                                   1 if causal else 0, float(scale), _ptr(out), _ptr(lse), _stream(stream))
    _check("attn_sink_fwd_paged", rc)
    return out, lse


def attn_sink_bwd(q, k, v, sink, out, lse, dout, cu_seqlens_q, cu_seqlens_k, max_seqlen_q,
                  max_seqlen_k, win_first=0, win_last=0, causal=True, scale=0.0, dq=None, dk=None,
                  dv=None, dsink=None, stream=None):
    """Backward with the sink's gradient; returns (dq, dk, dv, dsink or None)."""
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _need(t, torch.bfloat16, n)
    _need(sink, torch.float32, "sink")
    _need(lse, torch.float32, "lse")
    tq, hq, d = q.shape
    hkv = k.shape[1]
    dq = _made(stream, torch.empty_like, q) if dq is None else dq
    dk = _made(stream, torch.empty_like, k) if dk is None else dk
    dv = _made(stream, torch.empty_like, v) if dv is None else dv
    if sink is not None and dsink is None:
        dsink = _made(stream, torch.empty_like, sink)
    rc = lib().attn_sink_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(sink), _ptr(out), _ptr(lse), _ptr(dout),
                             _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), cu_seqlens_q.numel() - 1, tq,
                             k.shape[0], hq, hkv, d, int(max_seqlen_q), int(max_seqlen_k), int(win_first),
                             int(win_last), 1 if causal else 0, float(scale), _ptr(dq), _ptr(dk),
                             _ptr(dv), _ptr(dsink), _stream(stream))
    _check("attn_sink_bwd", rc)
    return dq, dk, dv, dsink


# ---------------------------------------------------------------------------
# Entry points around the cache: rotary positions, drafted trees, accumulated
# weights and eviction.  Their tensors must share one CUDA device (the library
# launches on it, whatever the current device is) and have the sizes that the
# pointers' readers assume; both are checked here.  A small call costs more on
# the host than on the GPU, so each function first tests its usual arguments in one
# expression (_is) and only otherwise goes through _expect, which names the
# argument that is wrong.

_BF16, _I32, _F32 = torch.bfloat16, torch.int32, torch.float32


def _is(t, dtype, dev, shape):
    """Whether t is a contiguous CUDA tensor of this type, device index and shape."""
    return t.dtype is dtype and t.get_device() == dev and t.shape == shape and t.is_contiguous()


def _device(name, t):
    """Device index of the call's first tensor."""
    dev = t.get_device()
    if dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    return dev


def _expect(name, t, dtype, dev, shape, contiguous=True):
    """Type, device and shape of an argument; None in `shape` stands for any extent."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.get_device() != dev:
        raise TypeError(f"{name} is on {t.device}, the call's first tensor on cuda:{dev}")
    got = t.shape
    if len(got) != len(shape) or any(w is not None and w != g for w, g in zip(shape, got)):
        raise TypeError(f"{name} must have shape {shape}, got {tuple(got)}")
    if contiguous and not t.is_contiguous():
        raise TypeError(f"{name} must be contiguous")


def _expect_rows(name, t, dev, shape):
    """A (rows, heads, d) bf16 tensor whose heads are contiguous within a row;
    returns its row stride (0: contiguous)."""
    if t.dtype is not _BF16 or t.get_device() != dev or t.dim() != 3 or t.shape != shape:
        _expect(name, t, _BF16, dev, shape, contiguous=False)
    if t.is_contiguous():
        return 0
    _, heads, d = t.shape
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != d) or t.stride(0) < heads * d:
        raise TypeError(f"{name}: heads must be contiguous within a row and rows must not overlap")
    return t.stride(0)


def _expect_inv_freq(inv_freq, dev, d):
    if inv_freq.dtype is not torch.float64 or inv_freq.get_device() != dev or inv_freq.dim() != 1:
        _expect("inv_freq", inv_freq, torch.float64, dev, (None,))
    n = inv_freq.shape[0]
    if not 1 <= n <= d // 2:
        raise TypeError(f"inv_freq must hold 1 .. head_dim / 2 frequencies, got {n}")
    if not inv_freq.is_contiguous():
        raise TypeError("inv_freq must be contiguous")
    return 2 * n


def _expect_cache(k_cache, v_cache, page_table, dev, batch=None, d=None):
    """Returns (num_pages, page_size, hkv, d, max_pages)."""
    shape = k_cache.shape
    if len(shape) != 4 or (d is not None and shape[3] != d) or not _is(k_cache, _BF16, dev, shape):
        _expect("k_cache", k_cache, _BF16, dev, (None, None, None, d))
    if not _is(v_cache, _BF16, dev, shape):
        _expect("v_cache", v_cache, _BF16, dev, shape)
    if page_table.dim() != 2 or not _is(page_table, _I32, dev, (page_table.shape[0] if batch is None else batch,
                                                                page_table.shape[1])):
        _expect("page_table", page_table, _I32, dev, (batch, None))
    return (*shape, page_table.shape[1])


_entry = {}


def _run(name, dev, stream, *args):
    """Calls the entry point on device `dev` and `stream` (None: the device's current one)."""
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(lib(), name)
    raw = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, raw)
    if rc != OK:
        _check(name, rc)


def attn_sink_rope(q, k, positions, inv_freq, interleaved=False, attn_scale=1.0, inverse=False, q_out=None,
                   k_out=None, stream=None):
    """Rotary positions: rotates the first 2 * len(inv_freq) dimensions of every head
    of q (T, Hq, d) and k (T, Hkv, d, or None) by positions (T,) int32 times inv_freq
    (fp64, radians per position; see attn_sink_rope_freqs), by the negative angle
    with `inverse` (the gradient).  Rows may be strided (column ranges of a packed
    buffer); an output may be its own input.  Returns (q_out, k_out or None)."""
    dev = _device("q", q)
    q_rs = _expect_rows("q", q, dev, (None, None, None) if q.dim() != 3 else q.shape)
    T, hq, d = q.shape
    if not _is(positions, _I32, dev, (T,)):
        _expect("positions", positions, _I32, dev, (T,))
    r = _expect_inv_freq(inv_freq, dev, d)
    if q_out is None:
        q_out, qo_rs = _made(stream, torch.empty_like, q, memory_format=torch.contiguous_format), 0
    else:
        qo_rs = _expect_rows("q_out", q_out, dev, q.shape)
    hkv = k_rs = ko_rs = 0
    kp = kop = None
    if k is not None:
        k_rs = _expect_rows("k", k, dev, (T, None if k.dim() != 3 else k.shape[1], d))
        hkv = k.shape[1]
        if k_out is None:
            k_out = _made(stream, torch.empty_like, k, memory_format=torch.contiguous_format)
        else:
            ko_rs = _expect_rows("k_out", k_out, dev, k.shape)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise TypeError("k_out is given without k")
    _run("attn_sink_rope", dev, stream, q.data_ptr(), q_out.data_ptr(), kp, kop, q_rs, qo_rs, k_rs, ko_rs,
         positions.data_ptr(), inv_freq.data_ptr(), T, hq, hkv, d, r, 1 if interleaved else 0, 1 if inverse else 0,
         float(attn_scale))
    return q_out, k_out


def rope_checked(q, k, positions, inv_freq, interleaved, attn_scale, inverse):
    """attn_sink_rope for contiguous q and k (or None) whose forward call has passed its
    checks: the backward's call, which runs on autograd's thread, where the
    interpreter's time counts most."""
    T, hq, d = q.shape
    q_out = torch.empty_like(q)
    kp = kop = k_out = None
    hkv = 0
    if k is not None:
        k_out = torch.empty_like(k)
        hkv = k.shape[1]
        kp, kop = k.data_ptr(), k_out.data_ptr()
    _run("attn_sink_rope", q.get_device(), None, q.data_ptr(), q_out.data_ptr(), kp, kop, 0, 0, 0, 0,
         positions.data_ptr(), inv_freq.data_ptr(), T, hq, hkv, d, 2 * inv_freq.shape[0], 1 if interleaved else 0,
         1 if inverse else 0, attn_scale)
    return q_out, k_out


def attn_sink_rope_kv_append(q, k_new, v_new, k_cache, v_cache, page_table, seqlens, inv_freq, cu_new=None,
                             max_new=None, positions=None, interleaved=False, attn_scale=1.0, q_out=None,
                             stream=None):
    """Rotates the new tokens' q (T, Hq, d) into q_out, and k_new (T, Hkv, d) into the
    paged caches together with v_new, in one launch (see attn_sink_kv_append for the
    slots).  `positions` (T,) int32 defaults to each row's logical token.  Returns
    q_out, whose rows behind the last request's are left as they were (unset in a
    q_out that is allocated here)."""
    dev = _device("q", q)
    q_rs = _expect_rows("q", q, dev, (None, None, None) if q.dim() != 3 else q.shape)
    T, hq, d = q.shape
    B = seqlens.shape[0] if seqlens.dim() == 1 else None
    if B is None or not _is(seqlens, _I32, dev, (B,)):
        _expect("seqlens", seqlens, _I32, dev, (None,))
    npages, ps, hkv, _, max_pages = _expect_cache(k_cache, v_cache, page_table, dev, B, d)
    k_rs = _expect_rows("k_new", k_new, dev, (T, hkv, d))
    v_rs = _expect_rows("v_new", v_new, dev, (T, hkv, d))
    r = _expect_inv_freq(inv_freq, dev, d)
    cu = pos = None
    if cu_new is None:
        if T != B:
            raise TypeError(f"without cu_new every request has one new row: got {T} rows, {B} requests")
        max_new = 1 if max_new is None else max_new
    else:
        if not _is(cu_new, _I32, dev, (B + 1,)):
            _expect("cu_new", cu_new, _I32, dev, (B + 1,))
        cu = cu_new.data_ptr()
        if max_new is None:
            max_new = int((cu_new[1:] - cu_new[:-1]).max()) if B else 0
    if positions is not None:
        if not _is(positions, _I32, dev, (T,)):
            _expect("positions", positions, _I32, dev, (T,))
        pos = positions.data_ptr()
    if q_out is None:
        q_out, qo_rs = _made(stream, torch.empty_like, q, memory_format=torch.contiguous_format), 0
    else:
        qo_rs = _expect_rows("q_out", q_out, dev, q.shape)
    _run("attn_sink_rope_kv_append", dev, stream, q.data_ptr(), q_out.data_ptr(), k_new.data_ptr(), v_new.data_ptr(),
         q_rs, qo_rs, k_rs, v_rs, cu, pos, inv_freq.data_ptr(), seqlens.data_ptr(), page_table.data_ptr(), max_pages, B,
         T, hq, hkv, d, r, ps, npages, int(max_new), 1 if interleaved else 0, float(attn_scale), k_cache.data_ptr(),
         v_cache.data_ptr())
    return q_out


def _outputs(q, dev, lse_shape, sink, out, lse, return_lse, stream):
    """Checks or makes the outputs of an attention call; returns them and the pointers
    of sink, out and lse."""
    hq = q.shape[1]
    if sink is not None and not _is(sink, _F32, dev, (hq,)):
        _expect("sink", sink, _F32, dev, (hq,))
    if out is None:
        out = _made(stream, torch.empty_like, q)
    elif not _is(out, _BF16, dev, q.shape):
        _expect("out", out, _BF16, dev, q.shape)
    if lse is not None:
        if not _is(lse, _F32, dev, lse_shape):
            _expect("lse", lse, _F32, dev, lse_shape)
    elif return_lse:
        lse = _made(stream, torch.empty, lse_shape, dtype=_F32, device=q.device)
    return (out, lse, None if sink is None else sink.data_ptr(), out.data_ptr(),
            None if lse is None else lse.data_ptr())


def attn_sink_tree_paged(q, k_cache, v_cache, page_table, cu_seqlens_q, seqlens_k, parents, max_seqlen_q,
                         max_seqlen_k, sink=None, win_first=0, win_last=0, scale=0.0, out=None, lse=None,
                         return_lse=True, stream=None):
    """Attention of trees of drafted tokens (at most 256 a request) over a paged cache
    that holds their K/V.  q (T, Hq, d); parents (T,) int32: the node's parent as an
    index in its request, -1 on the prefix.  Returns (out, lse (Hq, T))."""
    dev = _device("q", q)
    if q.dim() != 3 or not _is(q, _BF16, dev, q.shape):
        _expect("q", q, _BF16, dev, (None, None, None))
    T, hq, d = q.shape
    B = seqlens_k.shape[0] if seqlens_k.dim() == 1 else None
    if B is None or not _is(seqlens_k, _I32, dev, (B,)):
        _expect("seqlens_k", seqlens_k, _I32, dev, (None,))
    npages, ps, hkv, _, max_pages = _expect_cache(k_cache, v_cache, page_table, dev, B, d)
    if not _is(cu_seqlens_q, _I32, dev, (B + 1,)):
        _expect("cu_seqlens_q", cu_seqlens_q, _I32, dev, (B + 1,))
    if not _is(parents, _I32, dev, (T,)):
        _expect("parents", parents, _I32, dev, (T,))
    out, lse, sp, op, lp = _outputs(q, dev, (hq, T), sink, out, lse, return_lse, stream)
    _run("attn_sink_tree_paged", dev, stream, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
         page_table.data_ptr(), max_pages, cu_seqlens_q.data_ptr(), seqlens_k.data_ptr(), parents.data_ptr(), B, T, hq,
         hkv, d, ps, npages, int(max_seqlen_q), int(max_seqlen_k), sp, int(win_first), int(win_last), float(scale), op,
         lp)
    return out, lse


def attn_sink_kv_compact(k_cache, v_cache, page_table, src, counts, base=None, stream=None):
    """Moves cached rows in place: token src[b, (h,) j] of request b becomes its token
    base[b] + j (base None: j) for j < counts[b].  src (B, m) or (B, Hkv, m) int32,
    increasing, src[j] >= base + j.  Returns (k_cache, v_cache)."""
    dev = _device("k_cache", k_cache)
    npages, ps, hkv, d, max_pages = _expect_cache(k_cache, v_cache, page_table, dev)
    B, shared = page_table.shape[0], src.dim() == 2
    most = src.shape[-1] if src.dim() else None
    want = (B, most) if shared else (B, hkv, most)
    if not _is(src, _I32, dev, want):
        _expect("src", src, _I32, dev, want)
    if not _is(counts, _I32, dev, (B,)):
        _expect("counts", counts, _I32, dev, (B,))
    bp = None
    if base is not None:
        if not _is(base, _I32, dev, (B,)):
            _expect("base", base, _I32, dev, (B,))
        bp = base.data_ptr()
    _run("attn_sink_kv_compact", dev, stream, k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), max_pages,
         src.data_ptr(), counts.data_ptr(), bp, B, 1 if shared else hkv, most, hkv, d, ps, npages)
    return k_cache, v_cache


def attn_sink_decode_paged_weights(q, k_cache, v_cache, page_table, seqlens, weights, sink=None, win_first=0,
                                   win_last=0, scale=0.0, out=None, lse=None, return_lse=True, stream=None,
                                   max_seqlen=None):
    """attn_sink_decode_paged that also adds every visible token's attention weight to
    weights (B, Hkv or 1, cap) fp32, summed over the query heads of the KV head (or
    all).  max_seqlen: a host bound of seqlens, worth giving where page_table is much wider
    than the requests are long (it sizes scratch and launches).  Returns (out, lse)."""
    dev = _device("q", q)
    if q.dim() != 3 or not _is(q, _BF16, dev, q.shape):
        _expect("q", q, _BF16, dev, (None, None, None))
    B, hq, d = q.shape
    npages, ps, hkv, _, max_pages = _expect_cache(k_cache, v_cache, page_table, dev, B, d)
    if not _is(seqlens, _I32, dev, (B,)):
        _expect("seqlens", seqlens, _I32, dev, (B,))
    shape = weights.shape
    if len(shape) != 3 or shape[0] != B or not _is(weights, _F32, dev, shape):
        _expect("weights", weights, _F32, dev, (B, None, None))
    out, lse, sp, op, lp = _outputs(q, dev, (B, hq), sink, out, lse, return_lse, stream)
    rest = (sp, int(win_first), int(win_last), float(scale), weights.data_ptr(), shape[1], shape[2], op, lp)
    sizes = (page_table.data_ptr(), max_pages, seqlens.data_ptr(), B, hq, hkv, d, ps, npages)
    if max_seqlen is None:
        _run("attn_sink_decode_paged_weights", dev, stream, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
             *sizes, *rest)
    else:
        _run("attn_sink_decode_paged_weights_bounded", dev, stream, q.data_ptr(), k_cache.data_ptr(),
             v_cache.data_ptr(), *sizes, min(int(max_seqlen), 2 ** 31 - 1), *rest)
    return out, lse


def attn_sink_evict_paged(k_cache, v_cache, page_table, seqlens, weights, budget, keep_first=0, keep_last=0,
                          weights_out=None, kept=None, new_seqlens=None, stream=None):
    """Brings every request with more than `budget` cached tokens down to it: kept are
    the first keep_first, the last keep_last and the others of largest weight
    (ties: the earlier token), moved to the front in their order, in place; weights
    (B, Hkv or 1, cap) fp32 follow them (into weights_out if given) and are 0 behind.
    Returns (new_seqlens (B,), kept (B, Hkv or 1, budget), -1 padded)."""
    dev = _device("k_cache", k_cache)
    npages, ps, hkv, d, max_pages = _expect_cache(k_cache, v_cache, page_table, dev)
    B = page_table.shape[0]
    if not _is(seqlens, _I32, dev, (B,)):
        _expect("seqlens", seqlens, _I32, dev, (B,))
    shape = weights.shape
    if len(shape) != 3 or shape[0] != B or not _is(weights, _F32, dev, shape):
        _expect("weights", weights, _F32, dev, (B, None, None))
    _, heads, cap = shape
    budget = int(budget)
    if weights_out is None:
        weights_out = weights
    elif not _is(weights_out, _F32, dev, shape):
        _expect("weights_out", weights_out, _F32, dev, shape)
    if kept is None:
        kept = _made(stream, torch.empty, (B, heads, max(budget, 0)), dtype=_I32, device=seqlens.device)
    elif not _is(kept, _I32, dev, (B, heads, budget)):
        _expect("kept", kept, _I32, dev, (B, heads, budget))
    if new_seqlens is None:
        new_seqlens = _made(stream, torch.empty_like, seqlens)
    elif not _is(new_seqlens, _I32, dev, (B,)):
        _expect("new_seqlens", new_seqlens, _I32, dev, (B,))
    _run("attn_sink_evict_paged", dev, stream, k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), max_pages,
         seqlens.data_ptr(), weights.data_ptr(), B, heads, cap, hkv, d, ps, npages, budget,
         int(keep_first), int(keep_last), weights_out.data_ptr(), kept.data_ptr(), new_seqlens.data_ptr())
    return new_seqlens, kept


def attn_sink_visible_ranges(seqlens, win_first, win_last, stream=None):
    _need(seqlens, torch.int32, "seqlens")
    B = seqlens.numel()
    ranges = _made(stream, torch.empty, (B, 4), dtype=torch.int32, device=seqlens.device)
    rc = lib().attn_sink_visible_ranges(_ptr(seqlens), B, int(win_first), int(win_last),
                                        _ptr(ranges), _stream(stream))
    _check("attn_sink_visible_ranges", rc)
    return ranges


def attn_sink_visible_slots(seqlens, page_table, page_size, num_pages, win_first, win_last,
                            max_visible, stream=None):
    _need(seqlens, torch.int32, "seqlens")
    _need(page_table, torch.int32, "page_table")
    B = seqlens.numel()
    slots = _made(stream, torch.empty, (B, max_visible), dtype=torch.int32, device=seqlens.device)
    rc = lib().attn_sink_visible_slots(_ptr(seqlens), _ptr(page_table), page_table.shape[1], B,
                                       int(page_size), int(num_pages), int(win_first),
                                       int(win_last), _ptr(slots), int(max_visible),
                                       _stream(stream))
    _check("attn_sink_visible_slots", rc)
    return slots


def attn_sink_selftest_wait(complete, stream=None):
    """One single-thread kernel waits on an mbarrier: completed first (returns at
    once) or never completed (gives up after the wait limit and sets DEV_TIMEOUT,
    read by device_status)."""
    _check("attn_sink_selftest_wait", lib().attn_sink_selftest_wait(1 if complete else 0, _stream(stream)))


def device_status(stream=None) -> int:
    rc = lib().attn_sink_device_status(_stream(stream))
    if rc < 0:
        _check("attn_sink_device_status", rc)
    return rc
