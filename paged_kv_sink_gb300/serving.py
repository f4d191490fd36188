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
    fmt, shape = _FORMATS.get(k_cache.dtype), k_cache.shape
    if fmt is None:
        raise TypeError(f"k_cache must be torch.float8_e4m3fn or torch.int8, got {k_cache.dtype}")
    if len(shape) != 4 or (d is not None and shape[3] != d) or not _is(k_cache, k_cache.dtype, dev, shape):
        _expect("k_cache", k_cache, k_cache.dtype, dev, (None, None, None, d))
    if not _is(v_cache, k_cache.dtype, dev, shape):
        _expect("v_cache", v_cache, k_cache.dtype, dev, shape)
    npages, ps, hkv, d = shape
    blocks = k_scale.shape[1] if k_scale.dim() == 3 else 0
    want = (npages, blocks, hkv)
    if not _is(k_scale, _F32, dev, want):
        _expect("k_scale", k_scale, _F32, dev, (npages, None, hkv))
    if not _is(v_scale, _F32, dev, want):
        _expect("v_scale", v_scale, _F32, dev, want)
    if blocks < 1 or ps % blocks:
        raise TypeError(f"k_scale has {blocks} blocks a page, which must divide its {ps} tokens")
    if page_table.dim() != 2 or not _is(page_table, _I32, dev, (batch, page_table.shape[1])):
        _expect("page_table", page_table, _I32, dev, (batch, None))
    return npages, ps, hkv, d, page_table.shape[1], ps // blocks, fmt


def _expect_i32(name, t, dev, n=None):
    if t.dim() != 1 or not _is(t, _I32, dev, (t.shape[0] if n is None else n,)):
        _expect(name, t, _I32, dev, (n,))
    return t.shape[0]


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
    (attn_sink_kv_append_q8): one to many query rows a request.  Returns (out, lse (Hq, T))."""
    dev = _device("q", q)
    if q.dim() != 3 or not _is(q, _BF16, dev, q.shape):
        _expect("q", q, _BF16, dev, (None, None, None))
    T, hq, d = q.shape
    B = _expect_i32("seqlens_k", seqlens_k, dev)
    npages, ps, hkv, _, max_pages, block, fmt = _expect_q8(k_cache, v_cache, k_scale, v_scale, page_table, dev, B, d)
    _expect_i32("cu_seqlens_q", cu_seqlens_q, dev, B + 1)
    out, lse, sp, op, lp = _outputs(q, dev, (hq, T), sink, out, lse, return_lse, stream)
    _run("attn_sink_fwd_paged_q8", dev, stream, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
         v_scale.data_ptr(), block, fmt, page_table.data_ptr(), max_pages, cu_seqlens_q.data_ptr(), seqlens_k.data_ptr(), B,
         T, hq, hkv, d, ps, npages, int(max_seqlen_q), int(max_seqlen_k), sp, int(win_first), int(win_last),
         1 if causal else 0, float(scale), op, lp)
    return out, lse


def _expect_probs(name, t, dtype, dev, shape):
    """A (rows, vocab) matrix with contiguous rows; returns its row stride."""
    if t.dtype != dtype or t.get_device() != dev or t.dim() != 2 or t.shape != shape:
        _expect(name, t, dtype, dev, shape, contiguous=False)
    rows, vocab = t.shape
    if vocab > 1 and t.stride(1) != 1 or rows > 1 and t.stride(0) < vocab:
        raise TypeError(f"{name}: a row's probabilities must be contiguous and rows must not overlap")
    return t.stride(0) if rows > 1 else 0


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
    dtype = _TYPES.get(target.dtype)
    if dtype is None:
        raise TypeError(f"target must be torch.float32, torch.bfloat16 or torch.float16, got {target.dtype}")
    shape = target.shape if target.dim() == 2 else (None, None)
    p_rs = _expect_probs("target", target, target.dtype, dev, shape)
    T, vocab = shape
    q_rs, qp = 0, None
    if draft is not None:
        q_rs, qp = _expect_probs("draft", draft, target.dtype, dev, shape), draft.data_ptr()
    B = _expect_i32("cu_seqlens", cu_seqlens, dev) - 1
    if B < 0:
        raise TypeError("cu_seqlens must have a number more than there are requests")
    _expect_i32("tokens", tokens, dev, T)
    if parents is not None:
        _expect_i32("parents", parents, dev, T)
    if base is not None:
        _expect_i32("base", base, dev, B)
    for name, t, n in (("u", u, T), ("u_next", u_next, B)):
        if not _is(t, _F32, dev, (n,)):
            _expect(name, t, _F32, dev, (n,))
    max_nodes = int(max_nodes)
    made = []
    for name, t, want in (("src", src, (B, max(max_nodes, 0))), ("counts", counts, (B,)),
                          ("next_tokens", next_tokens, (B,))):
        if t is None:
            t = _made(stream, torch.empty, want, dtype=_I32, device=target.device)
        elif not _is(t, _I32, dev, want):
            _expect(name, t, _I32, dev, want)
        made.append(t)
    _run("attn_sink_verify_draft", dev, stream, target.data_ptr(), qp, p_rs, q_rs, dtype, tokens.data_ptr(),
         None if parents is None else parents.data_ptr(), cu_seqlens.data_ptr(), u.data_ptr(), u_next.data_ptr(),
         None if base is None else base.data_ptr(), B, T, max_nodes, vocab, *(t.data_ptr() for t in made))
    return tuple(made)


def _expect_pools(caches, dev, num_pages):
    """The host arrays of the tensors' addresses and page sizes."""
    caches = (caches,) if isinstance(caches, torch.Tensor) else tuple(caches)
    for i, c in enumerate(caches):
        if c.get_device() != dev or not c.is_contiguous() or c.dim() < 2 or c.shape[0] != num_pages:
            _expect(f"caches[{i}]", c, c.dtype, dev, (num_pages,) + (None,) * max(1, c.dim() - 1))
    n = len(caches)
    ptrs = (ctypes.c_void_p * n)(*(c.data_ptr() for c in caches))
    sizes = (ctypes.c_longlong * n)(*(c.nbytes // num_pages if num_pages else 0 for c in caches))
    return ptrs, sizes, n


def _expect_table(page_table, refs, seqlens):
    """Returns (device, batch, max_pages, num_pages)."""
    dev = _device("page_table", page_table)
    if page_table.dim() != 2 or not _is(page_table, _I32, dev, page_table.shape):
        _expect("page_table", page_table, _I32, dev, (None, None))
    B, max_pages = page_table.shape
    n = _expect_i32("refs", refs, dev)
    _expect_i32("seqlens", seqlens, dev, B)
    return dev, B, max_pages, n


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
    if out_table is None:
        out_table = _made(stream, torch.empty, (n, max_pages), dtype=_I32, device=page_table.device)
    elif not _is(out_table, _I32, dev, (n, max_pages)):
        _expect("out_table", out_table, _I32, dev, (n, max_pages))
    if out_seqlens is None:
        out_seqlens = _made(stream, torch.empty, (n,), dtype=_I32, device=page_table.device)
    else:
        _expect_i32("out_seqlens", out_seqlens, dev, n)
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
    if missing is None:
        missing = _made(stream, torch.empty, (1,), dtype=_I32, device=page_table.device)
    else:
        _expect_i32("missing", missing, dev, 1)
    _run("attn_sink_pages_reserve", dev, stream, ptrs, sizes, n, page_table.data_ptr(), refs.data_ptr(),
         seqlens.data_ptr(), new_seqlens.data_ptr(), B, max_pages, int(page_size), pages, missing.data_ptr())
    return missing


def attn_sink_pages_compact(caches, page_table, refs, seqlens, page_size, held=None, stream=None):
    """Brings the held pages to the front of every tensor of ``caches``, with page_table and refs.
    Returns held (1,) int32, their number: the pages from there on are free."""
    dev, B, max_pages, pages = _expect_table(page_table, refs, seqlens)
    ptrs, sizes, n = _expect_pools(caches, dev, pages)
    if held is None:
        held = _made(stream, torch.empty, (1,), dtype=_I32, device=page_table.device)
    else:
        _expect_i32("held", held, dev, 1)
    _run("attn_sink_pages_compact", dev, stream, ptrs, sizes, n, page_table.data_ptr(), refs.data_ptr(),
         seqlens.data_ptr(), B, max_pages, int(page_size), pages, held.data_ptr())
    return held
