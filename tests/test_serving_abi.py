"""Refusals of the 8-bit cache's, the verification's and the pages' entry points (CPU: status codes
before any CUDA call, and the binding's checks)."""
import ctypes

import pytest
import torch

P, Q, R, S = (ctypes.c_void_p(16 * i) for i in (1, 2, 3, 4))  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(24)


@pytest.fixture(scope="module")
def lib():
    from paged_kv_sink_gb300 import build as b
    path = b.build()
    from paged_kv_sink_gb300 import _lib
    return _lib.load(path)


def append(lib, k=P, rs=(0, 0), cu=P, sl=P, pt=P, mp=4, batch=2, total=4, hkv=2, d=64, ps=16, np_=8, mx=2, block=16, fmt=0, kc=P,
           vc=Q, ks=R, vs=S):
    return lib.attn_sink_kv_append_q8(k, k, *rs, cu, sl, pt, mp, batch, total, hkv, d, ps, np_, mx, block, fmt, kc, vc, ks, vs, None)


@pytest.mark.parametrize("kw,rc,text", [
    (dict(d=96), -2, b"head_dim"), (dict(hkv=0), -1, b"sizes"), (dict(batch=-1), -1, b"sizes"), (dict(total=-1), -1, b"sizes"),
    (dict(mx=-1), -1, b"sizes"), (dict(block=0), -1, b"block"), (dict(block=5), -1, b"block"), (dict(block=32), -1, b"block"),
    (dict(fmt=2), -1, b"format"), (dict(fmt=-1), -1, b"format"), (dict(np_=1 << 28), -2, b"int32"), (dict(mp=(1 << 27) - 1), -2, b"int32"),
    (dict(kc=None), -1, b"NULL"), (dict(ks=None), -1, b"NULL"), (dict(sl=None), -1, b"NULL"), (dict(k=None), -1, b"NULL"),
    (dict(kc=ODD), -1, b"aligned"), (dict(k=ODD), -1, b"aligned"), (dict(vc=P), -1, b"differ"), (dict(vs=R), -1, b"differ"),
    (dict(rs=(100, 0)), -1, b"k_new row stride"), (dict(rs=(0, 132)), -1, b"v_new row stride"), (dict(cu=None), -1, b"cu_new"),
    (dict(cu=None, mx=1, total=1), -1, b"cu_new"), (dict(batch=65536), -2, b"batch"), (dict(hkv=65536), -2, b"hkv"),
    (dict(batch=0, k=None), 0, b""), (dict(mx=0, kc=None), 0, b""), (dict(total=0, k=None), 0, b""),
    (dict(batch=-1, mx=0), -1, b"sizes")])
def test_append_refusals(lib, kw, rc, text):
    assert append(lib, **kw) == rc and text in lib.attn_sink_last_error()


def decode(lib, q=P, kc=P, vc=Q, ks=R, vs=S, block=16, fmt=0, pt=P, mp=4, sl=P, batch=2, hq=8, hkv=2, d=64, ps=16, np_=8, most=64,
           wf=0, out=P):
    return lib.attn_sink_decode_paged_q8(q, kc, vc, ks, vs, block, fmt, pt, mp, sl, batch, hq, hkv, d, ps, np_, most, None, wf, 0, 0.0,
                                         out, None, None)


@pytest.mark.parametrize("kw,rc,text", [
    (dict(d=256), -2, b"head_dim"), (dict(hq=9), -2, b"hkv"), (dict(hq=0), -1, b"sizes"), (dict(wf=-1), -1, b"sizes"),
    (dict(most=-1), -1, b"sizes"), (dict(block=3), -1, b"block"), (dict(fmt=7), -1, b"format"), (dict(q=None), -1, b"NULL"),
    (dict(out=None), -1, b"NULL"), (dict(sl=None), -1, b"NULL"), (dict(vs=None), -1, b"NULL"), (dict(out=ODD), -1, b"aligned"),
    (dict(vc=ODD), -1, b"aligned"), (dict(batch=65536), -2, b"batch"), (dict(mp=0), -1, b"sizes"), (dict(batch=0, q=None), 0, b""),
    (dict(hq=32 * 65537, hkv=65536), -2, b"hkv")])
def test_decode_refusals(lib, kw, rc, text):
    assert decode(lib, **kw) == rc and text in lib.attn_sink_last_error()


def extend(lib, q=P, kc=P, vc=Q, block=16, fmt=1, mp=4, cu=P, batch=2, total=8, hq=8, hkv=2, d=64, ps=16, np_=8, mq=4, mk=64, wf=0,
           wl=0, causal=1, out=P):
    return lib.attn_sink_fwd_paged_q8(q, kc, vc, R, S, block, fmt, P, mp, cu, P, batch, total, hq, hkv, d, ps, np_, mq, mk, None, wf,
                                      wl, causal, 0.0, out, None, None)


@pytest.mark.parametrize("kw,rc,text", [
    (dict(d=32), -2, b"head_dim"), (dict(hq=9), -2, b"hkv"), (dict(mq=-1), -1, b"sizes"), (dict(mk=-1), -1, b"sizes"),
    (dict(total=-1), -1, b"sizes"), (dict(wf=-1), -1, b"sizes"), (dict(wl=4, causal=0), -1, b"causal"), (dict(block=7), -1, b"block"),
    (dict(fmt=2), -1, b"format"), (dict(cu=None), -1, b"NULL"), (dict(out=None), -1, b"NULL"), (dict(q=ODD), -1, b"aligned"),
    (dict(batch=65536), -2, b"batch"), (dict(mq=65535 * 128 + 1), -2, b"query rows"), (dict(batch=0, q=None), 0, b""),
    (dict(total=0, q=None), 0, b""), (dict(mq=0, q=None), 0, b"")])
def test_extend_refusals(lib, kw, rc, text):
    assert extend(lib, **kw) == rc and text in lib.attn_sink_last_error()


def verify(lib, p=P, q=Q, rs=(0, 0), dtype=0, tok=P, cu=P, u=P, un=P, batch=2, total=8, nodes=4, vocab=100, src=P, counts=Q, nxt=R):
    return lib.attn_sink_verify_draft(p, q, *rs, dtype, tok, None, cu, u, un, None, batch, total, nodes, vocab, src, counts, nxt, None)


@pytest.mark.parametrize("kw,rc,text", [
    (dict(batch=-1), -1, b"sizes"), (dict(total=-1), -1, b"sizes"), (dict(nodes=-1), -1, b"sizes"), (dict(vocab=0), -1, b"sizes"),
    (dict(dtype=3), -1, b"dtype"), (dict(nodes=257), -2, b"256"), (dict(vocab=1 << 20), -2, b"2^20"), (dict(rs=(99, 0)), -1, b"stride"),
    (dict(rs=(0, 99)), -1, b"stride"), (dict(rs=(-1, 0)), -1, b"stride"), (dict(p=None), -1, b"NULL"), (dict(tok=None), -1, b"NULL"),
    (dict(cu=None), -1, b"NULL"), (dict(u=None), -1, b"NULL"), (dict(un=None), -1, b"NULL"), (dict(src=None), -1, b"NULL"),
    (dict(counts=None), -1, b"NULL"), (dict(nxt=None), -1, b"NULL"), (dict(p=ctypes.c_void_p(18)), -1, b"aligned"),
    (dict(q=ctypes.c_void_p(17), dtype=1), -1, b"aligned"), (dict(batch=65536), -2, b"batch"), (dict(batch=0, p=None, cu=None), 0, b"")])
def test_verify_refusals(lib, kw, rc, text):
    assert verify(lib, **kw) == rc and text in lib.attn_sink_last_error()


def pools(*sizes, ptrs=None):
    n = len(sizes)
    return (ctypes.c_void_p * n)(*(ptrs or [16 * (i + 1) for i in range(n)])), (ctypes.c_longlong * n)(*sizes), n


def reserve(lib, name="reserve", pool=pools(64), table=P, refs=Q, sl=P, new=P, batch=2, mp=4, ps=16, np_=8, out=P):
    fn = getattr(lib, "attn_sink_pages_" + name)
    args = (table, refs, sl) if name == "compact" else (table, refs, sl, new)
    return fn(*pool, *args, batch, mp, ps, np_, out, None)


@pytest.mark.parametrize("name", ["reserve", "compact"])
@pytest.mark.parametrize("kw,rc,text", [
    (dict(batch=-1), -1, b"sizes"), (dict(ps=0), -1, b"sizes"), (dict(np_=0), -1, b"sizes"), (dict(table=None), -1, b"NULL"),
    (dict(refs=None), -1, b"NULL"), (dict(sl=None), -1, b"NULL"), (dict(out=None), -1, b"NULL"), (dict(batch=65536), -2, b"batch"),
    (dict(mp=(1 << 27) - 1), -2, b"int32"), (dict(pool=pools(*[16] * 9)), -2, b"8"), (dict(pool=pools(0)), -1, b"page_bytes"),
    (dict(pool=pools(-4)), -1, b"page_bytes"), (dict(pool=pools(4, 4, ptrs=[16, 16])), -1, b"differ"),
    (dict(pool=pools(4, ptrs=[None])), -1, b"NULL"), (dict(pool=(None, None, 2)), -1, b"NULL"), (dict(pool=(None, None, -1)), -1, b"sizes")])
def test_reserve_and_compact_refusals(lib, name, kw, rc, text):
    assert reserve(lib, name, **kw) == rc and text in lib.attn_sink_last_error()


def test_the_other_page_refusals(lib):
    err = lib.attn_sink_last_error
    copy = lambda pool=pools(64), np_=8, src=P, dst=P, n=3: lib.attn_sink_pages_copy(*pool, np_, src, dst, n, None)
    assert copy(n=-1) == -1 and copy(np_=0) == -1 and copy(src=None) == -1 and b"NULL" in err()
    assert copy(n=0, src=None) == 0
    fork = lambda t=P, r=Q, sl=R, src=P, b=2, ob=2, mp=4, ps=16, np_=8, ot=Q, os=S: lib.attn_sink_pages_fork(
        t, r, sl, src, b, ob, mp, ps, np_, ot, os, None)
    for kw, rc, text in ((dict(ob=-1), -1, b"sizes"), (dict(ob=65536), -2, b"batch"), (dict(b=65536), -2, b"batch"), (dict(ot=P), -1, b"inputs"),
                         (dict(os=R), -1, b"inputs"), (dict(src=None), -1, b"NULL"), (dict(t=None), -1, b"NULL"), (dict(r=None), -1, b"NULL"),
                         (dict(sl=None), -1, b"NULL"), (dict(ps=-1), -1, b"sizes")):
        assert fork(**kw) == rc and text in err(), kw
    release = lambda t=P, r=Q, sl=P, new=P, b=2, ps=16: lib.attn_sink_pages_release(t, r, sl, new, b, 4, ps, 8, None)
    for kw, rc, text in ((dict(new=None), -1, b"NULL"), (dict(sl=None), -1, b"NULL"), (dict(b=-1), -1, b"sizes"), (dict(ps=0), -1, b"sizes"),
                         (dict(b=0, t=None, new=None), 0, b"")):
        assert release(**kw) == rc and text in err(), kw


def test_binding_refuses_host_tensors(lib):
    import paged_kv_sink_gb300 as ext
    q, i, f = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    c, s, t = torch.zeros(4, 16, 2, 64, dtype=torch.int8), torch.zeros(4, 1, 2), torch.zeros(4, 1, dtype=torch.int32)
    for call in (lambda: ext.attn_sink_kv_append_q8(q, q, c, c, s, s, t, i), lambda: ext.attn_sink_decode_paged_q8(q, c, c, s, s, t, i),
                 lambda: ext.attn_sink_fwd_paged_q8(q, c, c, s, s, t, i, i, 1, 1), lambda: ext.attn_sink_verify_draft(s[0], i, None, i, f, f, 1),
                 lambda: ext.attn_sink_pages_copy([c], i, i), lambda: ext.attn_sink_pages_fork(t, i, i, i, 16),
                 lambda: ext.attn_sink_pages_release(t, i, i, i, 16), lambda: ext.attn_sink_pages_reserve([c], t, i, i, i, 16),
                 lambda: ext.attn_sink_pages_compact([c], t, i, i, 16)):
        with pytest.raises(TypeError, match="CUDA"):
            call()


@pytest.mark.gpu
def test_binding_checks_shapes(lib):
    import paged_kv_sink_gb300 as ext
    z = lambda *s, dtype=torch.int32: torch.zeros(*s, dtype=dtype, device="cuda")
    q, i, f = z(4, 2, 64, dtype=torch.bfloat16), z(4), z(4, dtype=torch.float32)
    c, s, t = z(4, 16, 2, 64, dtype=torch.int8), z(4, 1, 2, dtype=torch.float32), z(4, 1)
    c2, s2, p = c.clone(), s.clone(), z(4, 50, dtype=torch.float32)
    bad = [
        (lambda: ext.attn_sink_kv_append_q8(q, q, c.byte(), c2, s, s2, t, i), "float8_e4m3fn or torch.int8"),
        (lambda: ext.attn_sink_kv_append_q8(q, q, c, c2.view(torch.float8_e4m3fn), s, s2, t, i), "v_cache"),
        (lambda: ext.attn_sink_kv_append_q8(q, q, c, c2, s[:3], s2, t, i), "k_scale"),
        (lambda: ext.attn_sink_kv_append_q8(q, q, c, c2, z(4, 3, 2, dtype=torch.float32), z(4, 3, 2, dtype=torch.float32), t, i), "blocks"),
        (lambda: ext.attn_sink_kv_append_q8(q, q, c, c2, s, z(4, 2, 2, dtype=torch.float32), t, i), "v_scale"),
        (lambda: ext.attn_sink_kv_append_q8(q[:, :1], q, c, c2, s, s2, t, i), "k_new"),
        (lambda: ext.attn_sink_kv_append_q8(q[:3], q[:3], c, c2, s, s2, t, i), "cu_new"),
        (lambda: ext.attn_sink_kv_append_q8(q, q, c, c2, s, s2, t, i, cu_new=i), "cu_new"),
        (lambda: ext.attn_sink_decode_paged_q8(q, c, c2, s, s2, t[:2], i), "page_table"),
        (lambda: ext.attn_sink_decode_paged_q8(q, c, c2, s, s2, t, i[:2]), "seqlens"),
        (lambda: ext.attn_sink_decode_paged_q8(q, c, c2, s, s2, t, i, sink=f), "sink"),
        (lambda: ext.attn_sink_fwd_paged_q8(q, c, c2, s, s2, t, i, i, 1, 16), "cu_seqlens_q"),
        (lambda: ext.attn_sink_fwd_paged_q8(q, c, c2, s, s2, t, z(5), i, 1, 16, lse=f), "lse"),
        (lambda: ext.attn_sink_verify_draft(p.double(), i, None, z(3), f, f[:2], 2), "target"),
        (lambda: ext.attn_sink_verify_draft(p.t(), i, None, z(3), f, f[:2], 2), "contiguous"),
        (lambda: ext.attn_sink_verify_draft(p[:1].expand(4, 50), i, None, z(3), f, f[:2], 2), "overlap"),
        (lambda: ext.attn_sink_verify_draft(p, i, None, z(3), f, f[:2], 2, draft=p.half()), "draft"),
        (lambda: ext.attn_sink_verify_draft(p, i[:3], None, z(3), f, f[:2], 2), "tokens"),
        (lambda: ext.attn_sink_verify_draft(p, i, i[:2], z(3), f, f[:2], 2), "parents"),
        (lambda: ext.attn_sink_verify_draft(p, i, None, z(3), f, f, 2), "u_next"),
        (lambda: ext.attn_sink_verify_draft(p, i, None, z(0), f, f, 2), "cu_seqlens"),
        (lambda: ext.attn_sink_verify_draft(p, i, None, z(3), f, f[:2], 2, src=z(2, 3)), "src"),
        (lambda: ext.attn_sink_verify_draft(p, i, None, z(3), f, f[:2], 2, base=i), "base"),
        (lambda: ext.attn_sink_pages_copy([], i, i), "caches"), (lambda: ext.attn_sink_pages_copy([c, c2[:2]], i, i), "caches"),
        (lambda: ext.attn_sink_pages_copy([c], i, i[:2]), "dst"), (lambda: ext.attn_sink_pages_fork(t, i, i[:2], i, 16), "seqlens"),
        (lambda: ext.attn_sink_pages_fork(t, i, i, i, 16, out_table=z(4, 2)), "out_table"),
        (lambda: ext.attn_sink_pages_release(t, i, i, i[:2], 16), "new_seqlens"),
        (lambda: ext.attn_sink_pages_reserve([c.transpose(1, 2)], t, i, i, i, 16), "contiguous"),
        (lambda: ext.attn_sink_pages_reserve([c], t, i.long(), i, i, 16), "refs"),
        (lambda: ext.attn_sink_pages_compact([c], t, i, i, 16, held=z(2)), "held"),
    ]
    for call, word in bad:
        with pytest.raises(TypeError, match=word):
            call()
    for call in (lambda: ext.attn_sink_decode_paged_q8(q, c, c, s, s2, t, i), lambda: ext.attn_sink_verify_draft(p, i, None, z(3), f, f[:2], 300),
                 lambda: ext.attn_sink_pages_copy([c] * 2, i, i), lambda: ext.attn_sink_pages_fork(t, i, i, i, 0),
                 lambda: ext.attn_sink_pages_reserve([c.clone() for _ in range(9)], t, i, i, i, 16),
                 lambda: ext.attn_sink_decode_paged_q8(q, c, c2, s, s2, t, i, max_seqlen=-1)):
        with pytest.raises(ext.AttnSinkError):
            call()
