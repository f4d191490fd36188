"""Binding of what a server does with its cache next to attention: the 8-bit paged
cache, the verification of drafted tokens and the pages' bookkeeping (argument
marshalling only, as in _lib)."""
from __future__ import annotations

import ctypes

import torch

from ._lib import (_BF16, _F32, _I32, _device, _expect, _expect_rows, _is, _made, _outputs, _run)

__all__ = ["attn_sink_decode_paged_q8", "attn_sink_fwd_paged_q8", "attn_sink_kv_append_q8", "attn_sink_pages_compact",
           "attn_sink_pages_copy", "attn_sink_pages_fork", "attn_sink_pages_release", "attn_sink_pages_reserve",
           "attn_sink_verify_draft"]

_FORMATS = {torch.float8_e4m3fn: 0, torch.int8: 1}
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_NO_BOUND = 2 ** 31 - 1


def _expect_q8(k_cache, v_cache, k_scale, v_scale, page_table, dev, batch, d=None):
    """Returns (num_pages, page_size, hkv, d, max_pages, block, format)."""
    kind, shape, scales, table = k_cache.dtype, k_cache.shape, k_scale.shape, page_table.shape
    fmt = _FORMATS.get(kind)
    usual = (fmt is not None and len(shape) == 4 and len(scales) == 3 and len(table) == 2
             and (d is None or shape[3] == d) and _is(k_cache, kind, dev, shape) and _is(v_cache, kind, dev, shape)
             and scales[0] == shape[0] and scales[2] == shape[2] and _is(k_scale, _F32, dev, scales)
             and _is(v_scale, _F32, dev, scales) and table[0] == batch and _is(page_table, _I32, dev, table))
    if not usual:
        if fmt is None:
            raise TypeError(f"k_cache must be torch.float8_e4m3fn or torch.int8, got {kind}")
        _expect("k_cache", k_cache, kind, dev, (None, None, None, d))
        _expect("v_cache", v_cache, kind, dev, shape)
        _expect("k_scale", k_scale, _F32, dev, (shape[0], None, shape[2]))
        _expect("v_scale", v_scale, _F32, dev, scales)
        _expect("page_table", page_table, _I32, dev, (batch, None))
    blocks, ps = scales[1], shape[1]
    if blocks < 1 or ps % blocks:
        raise TypeError(f"k_scale has {blocks} blocks a page, which must divide its {ps} tokens")
    return shape[0], ps, shape[2], shape[3], table[1], ps // blocks, fmt


def _expect_i32(name, t, dev, n=None):
    """A (n,) int32 tensor (n None: of any length); returns its length."""
    shape = t.shape
    if len(shape) != 1 or (n is not None and shape[0] != n) or not _is(t, _I32, dev, shape):
        _expect(name, t, _I32, dev, (n,))
    return shape[0]


def attn_sink_kv_append_q8(k_new, v_new, k_cache, v_cache, k_scale, v_scale, page_table, seqlens, cu_new=None,
                           max_new=None, stream=None):
    """Writes the new K/V rows (T, Hkv, d) bf16 into an 8-bit paged cache in place.  Caches
    (P, ps, Hkv, d) torch.float8_e4m3fn or torch.int8; scales (P, blocks, Hkv) fp32, one for
    ps / blocks tokens of a KV head, powers of two (see the C header for how they grow).
    Rows may be strided (column ranges of a packed buffer).  Returns the caches and scales."""
    dev = _device("k_new", k_new)
    B = _expect_i32("seqlens", seqlens, dev)
    npages, ps, hkv, d, max_pages, block, fmt = _expect_q8(k_cache, v_cache, k_scale, v_scale, page_table, dev, B)
    T = k_new.shape[0] if k_new.dim() else None
    k_rs = _expect_rows("k_new", k_new, dev, (T, hkv, d))
    v_rs = _expect_rows("v_new", v_new, dev, (T, hkv, d))
    cu = None
    if cu_new is None:
        if T != B:
            raise TypeError(f"without cu_new every request has one new row: got {T} rows, {B} requests")
        max_new = 1 if max_new is None else max_new
    else:
        _expect_i32("cu_new", cu_new, dev, B + 1)
        cu = cu_new.data_ptr()
        if max_new is None:
            max_new = int((cu_new[1:] - cu_new[:-1]).max()) if B else 0
    _run("attn_sink_kv_append_q8", dev, stream, k_new.data_ptr(), v_new.data_ptr(), k_rs, v_rs, cu, seqlens.data_ptr(),
         page_table.data_ptr(), max_pages, B, T, hkv, d, ps, npages, int(max_new), block, fmt, k_cache.data_ptr(),
         v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr())
    return k_cache, v_cache, k_scale, v_scale


def attn_sink_decode_paged_q8(q, k_cache, v_cache, k_scale, v_scale, page_table, seqlens, sink=None, win_first=0,
                              win_last=0, scale=0.0, out=None, lse=None, return_lse=True, stream=None,
                              max_seqlen=None):
    """attn_sink_decode_paged over an 8-bit cache (see attn_sink_kv_append_q8).  max_seqlen: a
    host bound of seqlens, worth giving where page_table is much wider than the requests
    are long (it sizes scratch and launches).  Returns (out, lse)."""
    dev = _device("q", q)
    if q.dim() != 3 or not _is(q, _BF16, dev, q.shape):
        _expect("q", q, _BF16, dev, (None, None, None))
    B, hq, d = q.shape
    npages, ps, hkv, _, max_pages, block, fmt = _expect_q8(k_cache, v_cache, k_scale, v_scale, page_table, dev, B, d)
    _expect_i32("seqlens", seqlens, dev, B)
    out, lse, sp, op, lp = _outputs(q, dev, (B, hq), sink, out, lse, return_lse, stream)
    bound = _NO_BOUND if max_seqlen is None else min(int(max_seqlen), _NO_BOUND)
    _run("attn_sink_decode_paged_q8", dev, stream, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
         k_scale.data_ptr(), v_scale.data_ptr(), block, fmt, page_table.data_ptr(), max_pages, seqlens.data_ptr(), B, hq,
         hkv, d, ps, npages, bound, sp, int(win_first), int(win_last), float(scale), op, lp)
    return out, lse


def attn_sink_fwd_paged_q8(q, k_cache, v_cache, k_scale, v_scale, page_table, cu_seqlens_q, seqlens_k, max_seqlen_q,
                           max_seqlen_k, sink=None, win_first=0, win_last=0, causal=True, scale=0.0, out=None, lse=None,
                           return_lse=True, stream=None):
    """attn_sink_fwd_paged over an 8-bit cache that has the chunk's tokens already
    (attn_sink_kv_append_q8): one to many query rows a request.  max_seqlen_q and max_seqlen_k are
    host bounds of the rows and lengths.  Returns (out, lse (Hq, T))."""
    dev = _device("q", q)
    if q.dim() != 3 or not _is(q, _BF16, dev, q.shape):
        _expect("q", q, _BF16, dev, (None, None, None))
    T, hq, d = q.shape
    B = _expect_i32("seqlens_k", seqlens_k, dev)
    npages, ps, hkv, _, max_pages, block, fmt = _expect_q8(k_cache, v_cache, k_scale, v_scale, page_table, dev, B, d)
    _expect_i32("cu_seqlens_q", cu_seqlens_q, dev, B + 1)
    out, lse, sp, op, lp = _outputs(q, dev, (hq, T), sink, out, lse, return_lse, stream)
    max_seqlen_q, max_seqlen_k = min(int(max_seqlen_q), _NO_BOUND), min(int(max_seqlen_k), _NO_BOUND)
    _run("attn_sink_fwd_paged_q8", dev, stream, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
         v_scale.data_ptr(), block, fmt, page_table.data_ptr(), max_pages, cu_seqlens_q.data_ptr(), seqlens_k.data_ptr(), B,
         T, hq, hkv, d, ps, npages, max_seqlen_q, max_seqlen_k, sp, int(win_first), int(win_last),
         1 if causal else 0, float(scale), op, lp)
    return out, lse


def _row_stride(name, t):
    """Row stride of a (rows, vocab) matrix with contiguous rows (0: contiguous)."""
    if t.is_contiguous():
        return 0
    rows, vocab = t.shape
    if vocab > 1 and t.stride(1) != 1 or rows > 1 and t.stride(0) < vocab:
        raise TypeError(f"{name}: a row's probabilities must be contiguous and rows must not overlap")
    return t.stride(0) if rows > 1 else 0


def _output(name, t, like, shape, dev, stream):
    """An int32 output: checked, or made on the device of `like`."""
    if t is None:
        return like.new_empty(shape) if stream is None else _made(stream, like.new_empty, shape)
    if not _is(t, _I32, dev, shape):
        _expect(name, t, _I32, dev, shape)
    return t


def attn_sink_verify_draft(target, tokens, parents, cu_seqlens, u, u_next, max_nodes, draft=None, base=None, src=None,
                           counts=None, next_tokens=None, stream=None):
    """Verification of drafted tokens.  Request b's rows [cu_seqlens[b], cu_seqlens[b + 1]) are
    its last token (node 0) and its drafted ones; tokens (T,) int32, parents (T,) int32 (an
    earlier node of the request; None: the node before), target (T, vocab) fp32, bf16 or fp16:
    the target's probabilities of the token after each node, draft: the draft model's (None:
    the drafted tokens were chosen, not drawn).  u (T,) and u_next (B,) fp32 are random numbers
    in [0, 1).  Returns (src (B, max_nodes), counts (B,), next_tokens (B,)) int32: the nodes that
    stand as base[b] + index, -1 behind (attn_sink_kv_compact's src and counts, with base the
    prefix's length), their number, and the token that follows them."""
    dev = _device("target", target)
    kind, shape = target.dtype, target.shape
    dtype = _TYPES.get(kind)
    if dtype is None:
        raise TypeError(f"target must be torch.float32, torch.bfloat16 or torch.float16, got {kind}")
    if len(shape) != 2:
        _expect("target", target, kind, dev, (None, None))
    T, vocab = shape
    p_rs = _row_stride("target", target)
    q_rs, qp = 0, None
    if draft is not None:
        if draft.dtype != kind or draft.shape != shape or draft.get_device() != dev:
            _expect("draft", draft, kind, dev, tuple(shape), contiguous=False)
        q_rs, qp = _row_stride("draft", draft), draft.data_ptr()
    B = _expect_i32("cu_seqlens", cu_seqlens, dev) - 1
    if B < 0:
        raise TypeError("cu_seqlens must have a number more than there are requests")
    _expect_i32("tokens", tokens, dev, T)
    up = bp = None
    if parents is not None:
        _expect_i32("parents", parents, dev, T)
        up = parents.data_ptr()
    if base is not None:
        _expect_i32("base", base, dev, B)
        bp = base.data_ptr()
    if not _is(u, _F32, dev, (T,)):
        _expect("u", u, _F32, dev, (T,))
    if not _is(u_next, _F32, dev, (B,)):
        _expect("u_next", u_next, _F32, dev, (B,))
    max_nodes = int(max_nodes)
    src = _output("src", src, tokens, (B, max(max_nodes, 0)), dev, stream)
    counts = _output("counts", counts, tokens, (B,), dev, stream)
    next_tokens = _output("next_tokens", next_tokens, tokens, (B,), dev, stream)
    _run("attn_sink_verify_draft", dev, stream, target.data_ptr(), qp, p_rs, q_rs, dtype, tokens.data_ptr(), up,
         cu_seqlens.data_ptr(), u.data_ptr(), u_next.data_ptr(), bp, B, T, max_nodes, vocab, src.data_ptr(),
         counts.data_ptr(), next_tokens.data_ptr())
    return src, counts, next_tokens


_PTRS = [ctypes.c_void_p * n for n in range(9)]  # (a call has at most 8 tensors)
_SIZES = [ctypes.c_longlong * n for n in range(9)]


def _expect_pools(caches, dev, num_pages):
    """The host arrays of the tensors' addresses and page sizes."""
    if isinstance(caches, torch.Tensor):
        caches = (caches,)
    ptrs, sizes = [], []
    for i, c in enumerate(caches):
        shape = c.shape
        if len(shape) < 2 or shape[0] != num_pages or c.get_device() != dev or not c.is_contiguous():
            _expect(f"caches[{i}]", c, c.dtype, dev, (num_pages,) + (None,) * max(1, len(shape) - 1))
        ptrs.append(c.data_ptr())
        sizes.append(c.nbytes // num_pages if num_pages else 0)
    n = len(ptrs)
    if n > 8:
        return (ctypes.c_void_p * n)(*ptrs), (ctypes.c_longlong * n)(*sizes), n
    return _PTRS[n](*ptrs), _SIZES[n](*sizes), n


def _expect_table(page_table, refs, seqlens):
    """Returns (device, batch, max_pages, num_pages)."""
    dev, table, pool = _device("page_table", page_table), page_table.shape, refs.shape
    if not (len(table) == 2 and len(pool) == 1 and _is(page_table, _I32, dev, table) and _is(refs, _I32, dev, pool)
            and _is(seqlens, _I32, dev, table[:1])):
        _expect("page_table", page_table, _I32, dev, (None, None))
        _expect("refs", refs, _I32, dev, (None,))
        _expect("seqlens", seqlens, _I32, dev, (table[0],))
    return dev, table[0], table[1], pool[0]


def attn_sink_pages_copy(caches, src, dst, stream=None):
    """Copies page src[i] to page dst[i] in every tensor of ``caches`` (up to 8, pages along
    the first dimension; -1 for both: no copy).  No page may be written twice, or be written
    and read."""
    caches = (caches,) if isinstance(caches, torch.Tensor) else tuple(caches)
    if not caches:
        raise TypeError("caches must hold a tensor")
    dev = _device("caches[0]", caches[0])
    pages = caches[0].shape[0]
    ptrs, sizes, n = _expect_pools(caches, dev, pages)
    count = _expect_i32("src", src, dev)
    _expect_i32("dst", dst, dev, count)
    _run("attn_sink_pages_copy", dev, stream, ptrs, sizes, n, pages, src.data_ptr(), dst.data_ptr(), count)


def attn_sink_pages_fork(page_table, refs, seqlens, src, page_size, out_table=None, out_seqlens=None, stream=None):
    """A page table whose row b is row src[b] of ``page_table`` (-1: a row without tokens); refs
    (num_pages,), the number of entries that hold each page, follows in place.  Returns
    (table (len(src), max_pages), seqlens (len(src),))."""
    dev, B, max_pages, pages = _expect_table(page_table, refs, seqlens)
    n = _expect_i32("src", src, dev)
    out_table = _output("out_table", out_table, page_table, (n, max_pages), dev, stream)
    out_seqlens = _output("out_seqlens", out_seqlens, page_table, (n,), dev, stream)
    _run("attn_sink_pages_fork", dev, stream, page_table.data_ptr(), refs.data_ptr(), seqlens.data_ptr(), src.data_ptr(), B,
         n, max_pages, int(page_size), pages, out_table.data_ptr(), out_seqlens.data_ptr())
    return out_table, out_seqlens


def attn_sink_pages_release(page_table, refs, seqlens, new_seqlens, page_size, stream=None):
    """Gives back the pages of requests that shrink from seqlens to new_seqlens tokens (0: all
    of them), in page_table and refs in place."""
    dev, B, max_pages, pages = _expect_table(page_table, refs, seqlens)
    _expect_i32("new_seqlens", new_seqlens, dev, B)
    _run("attn_sink_pages_release", dev, stream, page_table.data_ptr(), refs.data_ptr(), seqlens.data_ptr(),
         new_seqlens.data_ptr(), B, max_pages, int(page_size), pages)


def attn_sink_pages_reserve(caches, page_table, refs, seqlens, new_seqlens, page_size, missing=None, stream=None):
    """Pages for requests that grow from seqlens to new_seqlens tokens: free ones, lowest first,
    and copies of partly filled pages that others hold too (in every tensor of ``caches``).
    Returns missing (1,) int32: 0, or the pages that are too few, and then nothing changed."""
    dev, B, max_pages, pages = _expect_table(page_table, refs, seqlens)
    _expect_i32("new_seqlens", new_seqlens, dev, B)
    ptrs, sizes, n = _expect_pools(caches, dev, pages)
    missing = _output("missing", missing, page_table, (1,), dev, stream)
    _run("attn_sink_pages_reserve", dev, stream, ptrs, sizes, n, page_table.data_ptr(), refs.data_ptr(),
         seqlens.data_ptr(), new_seqlens.data_ptr(), B, max_pages, int(page_size), pages, missing.data_ptr())
    return missing


def attn_sink_pages_compact(caches, page_table, refs, seqlens, page_size, held=None, stream=None):
    """Brings the held pages to the front of every tensor of ``caches``, with page_table and refs.
    Returns held (1,) int32, their number: the pages from there on are free."""
    dev, B, max_pages, pages = _expect_table(page_table, refs, seqlens)
    ptrs, sizes, n = _expect_pools(caches, dev, pages)
    held = _output("held", held, page_table, (1,), dev, stream)
    _run("attn_sink_pages_compact", dev, stream, ptrs, sizes, n, page_table.data_ptr(), refs.data_ptr(),
         seqlens.data_ptr(), B, max_pages, int(page_size), pages, held.data_ptr())
    return held
