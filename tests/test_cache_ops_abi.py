"""Refusals of the operators around the paged cache: status codes of the C entry
points before any CUDA call, and the binding's checks (CPU)."""
import ctypes

import pytest
import torch

P, Q = ctypes.c_void_p(16), ctypes.c_void_p(32)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(24)


@pytest.fixture(scope="module")
def lib():
    from paged_kv_sink_gb300 import build as b
    path = b.build()
    from paged_kv_sink_gb300 import _lib
    return _lib.load(path)


def rope(lib, q=P, q_out=P, k=Q, k_out=Q, rs=(0, 0, 0, 0), pos=P, f=P, rows=4, hq=8, hkv=2, d=64, r=64, m=1.0):
    return lib.attn_sink_rope(q, q_out, k, k_out, *rs, pos, f, rows, hq, hkv, d, r, 0, 0, m, None)


@pytest.mark.parametrize("kw,rc,text", [
    (dict(d=96), -2, b"head_dim"), (dict(r=0), -1, b"rotary_dim"), (dict(r=33), -1, b"rotary_dim"),
    (dict(r=66), -1, b"rotary_dim"), (dict(hq=0), -1, b"sizes"), (dict(rows=-1), -1, b"sizes"),
    (dict(hq=16384), -2, b"16384"), (dict(m=float("nan")), -1, b"attn_scale"), (dict(m=float("inf")), -1, b"attn_scale"),
    (dict(k=None), -1, b"together"), (dict(pos=None), -1, b"NULL"), (dict(f=None), -1, b"NULL"),
    (dict(q=ODD), -1, b"aligned"), (dict(k_out=ODD), -1, b"aligned"), (dict(rs=(100, 0, 0, 0)), -1, b"q row stride"),
    (dict(rs=(0, 0, 0, 132)), -1, b"k_out row stride"), (dict(rows=0, q=None), 0, b"")])
def test_rope_refusals(lib, kw, rc, text):
    assert rope(lib, **kw) == rc and text in lib.attn_sink_last_error()


def append(lib, q=P, k=P, kc=P, vc=Q, cu=P, rs=(0, 0, 0, 0), sl=P, pt=P, mp=4, batch=2, total=4, hq=8, hkv=2, d=64, r=64,
           ps=16, np_=8, max_new=2):
    return lib.attn_sink_rope_kv_append(q, q, k, k, *rs, cu, None, P, sl, pt, mp, batch, total, hq, hkv, d, r, ps, np_,
                                        max_new, 0, 1.0, kc, vc, None)


@pytest.mark.parametrize("kw,rc,text", [
    (dict(d=32), -2, b"head_dim"), (dict(r=1), -1, b"rotary_dim"), (dict(hkv=0), -1, b"sizes"),
    (dict(batch=-1), -1, b"sizes"), (dict(mp=0), -1, b"sizes"), (dict(np_=1 << 28), -2, b"int32"),
    (dict(max_new=-1), -1, b"max_new"), (dict(cu=None), -1, b"cu_new"), (dict(cu=None, max_new=1, total=1), -1, b"cu_new"),
    (dict(kc=None), -1, b"NULL"), (dict(vc=ODD), -1, b"aligned"), (dict(rs=(0, 0, 64, 0)), -1, b"k_new row stride"),
    (dict(batch=65536), -2, b"batch"), (dict(batch=0, q=None), 0, b""), (dict(max_new=0, q=None), 0, b"")])
def test_rope_append_refusals(lib, kw, rc, text):
    assert append(lib, **kw) == rc and text in lib.attn_sink_last_error()


def tree(lib, q=P, kc=P, cu=P, par=P, batch=2, total=8, hq=8, hkv=2, d=64, ps=16, np_=8, mq=4, mk=64, wf=0, out=P, mp=4):
    return lib.attn_sink_tree_paged(q, kc, kc, P, mp, cu, P, par, batch, total, hq, hkv, d, ps, np_, mq, mk, None, wf, 0,
                                    0.0, out, None, None)


@pytest.mark.parametrize("kw,rc,text", [
    (dict(d=256), -2, b"head_dim"), (dict(hq=9), -2, b"hkv"), (dict(hq=258, hkv=2), -2, b"hkv"),
    (dict(ps=24), -2, b"page_size"), (dict(ps=4), -2, b"page_size"), (dict(mq=257), -2, b"256"), (dict(mq=-1), -1, b"sizes"),
    (dict(wf=-1), -1, b"sizes"), (dict(par=None), -1, b"NULL"), (dict(out=None), -1, b"NULL"), (dict(q=ODD), -1, b"aligned"),
    (dict(batch=65536), -2, b"batch"), (dict(mp=0), -1, b"sizes"), (dict(batch=0, q=None), 0, b""),
    (dict(total=0, q=None), 0, b"")])
def test_tree_refusals(lib, kw, rc, text):
    assert tree(lib, **kw) == rc and text in lib.attn_sink_last_error()


def test_tree_refuses_a_negative_length_bound(lib):
    assert tree(lib, mk=-1) == -1 and b"sizes" in lib.attn_sink_last_error()
    assert tree(lib, mk=-2 ** 31) == -1 and tree(lib, mk=0, total=0) == 0


def compact(lib, kc=P, vc=Q, src=P, batch=2, heads=1, rows=4, hkv=2, d=64, ps=16, np_=8, mp=4):
    return lib.attn_sink_kv_compact(kc, vc, P, mp, src, P, None, batch, heads, rows, hkv, d, ps, np_, None)


@pytest.mark.parametrize("kw,rc,text", [
    (dict(d=96), -2, b"head_dim"), (dict(heads=3), -1, b"src_heads"), (dict(hkv=0), -1, b"sizes"), (dict(rows=-1), -1, b"sizes"),
    (dict(vc=P), -1, b"differ"), (dict(src=None), -1, b"NULL"), (dict(kc=ODD), -1, b"aligned"), (dict(batch=65536), -2, b"batch"),
    (dict(heads=40000, hkv=40000), -2, b"src_heads"), (dict(ps=0), -1, b"sizes"), (dict(rows=0, src=None), 0, b"")])
def test_compact_refusals(lib, kw, rc, text):
    assert compact(lib, **kw) == rc and text in lib.attn_sink_last_error()


def weights(lib, q=P, w=P, batch=2, hq=8, hkv=2, d=64, heads=2, cap=64):
    return lib.attn_sink_decode_paged_weights(q, P, P, P, 4, P, batch, hq, hkv, d, 16, 8, None, 0, 0, 0.0, w, heads, cap, P,
                                              None, None)


@pytest.mark.parametrize("kw,rc,text", [
    (dict(d=96), -2, b"head_dim"), (dict(heads=3), -1, b"weight_heads"), (dict(cap=-1), -1, b"weight_cap"),
    (dict(w=None), -1, b"weights"), (dict(hq=8192, hkv=64, heads=64), -2, b"4096"), (dict(q=ODD), -1, b"aligned"),
    (dict(batch=0, q=None), 0, b"")])
def test_weights_refusals(lib, kw, rc, text):
    assert weights(lib, **kw) == rc and text in lib.attn_sink_last_error()


@pytest.mark.parametrize("most,rc,text", [(-1, -1, b"max_seqlen"), (-2 ** 31, -1, b"max_seqlen"), (5, -1, b"weights")])
def test_bounded_weights_refusals(lib, most, rc, text):
    assert lib.attn_sink_decode_paged_weights_bounded(P, P, P, P, 4, P, 2, 8, 2, 64, 16, 8, most, None, 0, 0, 0.0, None, 2,
                                                      64, P, None, None) == rc
    assert text in lib.attn_sink_last_error()


@pytest.mark.parametrize("kw,rc,text", [
    (dict(hq=1024, hkv=1024, heads=1), -2, b"6144"), (dict(hq=4000, hkv=400, heads=1), -2, b"6144"),
    (dict(hq=4096, hkv=512, heads=1, w=None), -1, b"NULL")])
def test_weights_refuse_more_heads_than_one_accumulator_sums(lib, kw, rc, text):
    assert weights(lib, **kw) == rc and text in lib.attn_sink_last_error()


def test_requests_that_reach_the_end_of_int32_are_refused(lib):
    for call in (append, tree, compact):
        assert call(lib, mp=(1 << 27) - 1) == -2 and b"int32" in lib.attn_sink_last_error()


def evict(lib, kc=P, vc=Q, sl=P, batch=2, heads=1, cap=64, hkv=2, d=64, budget=16, first=1, last=2, new=Q, kept=P):
    return lib.attn_sink_evict_paged(kc, vc, P, 4, sl, P, batch, heads, cap, hkv, d, 16, 8, budget, first, last, P, kept,
                                     new, None)


@pytest.mark.parametrize("kw,rc,text", [
    (dict(d=96), -2, b"head_dim"), (dict(heads=4), -1, b"weight_heads"), (dict(cap=0), -1, b"sizes"),
    (dict(budget=0), -1, b"budget"), (dict(first=-1), -1, b"budget"), (dict(last=16), -1, b"budget"),
    (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), -1, b"budget"), (dict(vc=P), -1, b"differ"), (dict(new=P), -1, b"new_seqlens"),
    (dict(kept=None), -1, b"NULL"), (dict(vc=ODD), -1, b"aligned"), (dict(batch=65536), -2, b"batch"),
    (dict(batch=0, kc=None), 0, b"")])
def test_evict_refusals(lib, kw, rc, text):
    assert evict(lib, **kw) == rc and text in lib.attn_sink_last_error()


def test_binding_refuses_host_tensors_and_wrong_types(lib):
    import paged_kv_sink_gb300 as ext
    q, c = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, 16, 1, 64, dtype=torch.bfloat16)
    i, f, w = torch.zeros(4, dtype=torch.int32), torch.ones(32, dtype=torch.float64), torch.zeros(4, 1, 64)
    t = i[:, None].contiguous()
    for call in (lambda: ext.attn_sink_rope(q, None, i, f), lambda: ext.attn_sink_rope_func(q, q, i, f),
                 lambda: ext.attn_sink_rope_kv_append(q, q, q, c, c, t, i, f),
                 lambda: ext.attn_sink_tree_paged(q, c, c, t, i, i, i, 1, 1), lambda: ext.attn_sink_kv_compact(c, c, t, t, i),
                 lambda: ext.attn_sink_decode_paged_weights(q, c, c, t, i, w),
                 lambda: ext.attn_sink_evict_paged(c, c, t, i, w, 4)):
        with pytest.raises(TypeError, match="CUDA"):
            call()


@pytest.mark.gpu
def test_binding_checks_shapes(lib):
    import paged_kv_sink_gb300 as ext
    q, c = torch.zeros(4, 2, 64, dtype=torch.bfloat16).cuda(), torch.zeros(4, 16, 1, 64, dtype=torch.bfloat16).cuda()
    i, f = torch.zeros(4, dtype=torch.int32).cuda(), torch.ones(32, dtype=torch.float64).cuda()
    t, w, c2 = i[:, None].contiguous(), torch.zeros(4, 1, 64).cuda(), c.clone()
    bad = [
        (lambda: ext.attn_sink_rope(q, None, i[:3], f), "positions"), (lambda: ext.attn_sink_rope(q, None, i, f.float()), "inv_freq"),
        (lambda: ext.attn_sink_rope(q, None, i, torch.cat([f, f])), "frequencies"), (lambda: ext.attn_sink_rope(q, None, i, f[:0]), "frequencies"),
        (lambda: ext.attn_sink_rope(q[:1].expand(4, 2, 64), None, i, f), "overlap"),
        (lambda: ext.attn_sink_rope(q.transpose(0, 1), None, i[:2], f), "contiguous"),
        (lambda: ext.attn_sink_rope(q, None, i, f, k_out=q), "k_out"), (lambda: ext.attn_sink_rope(q, q[:3], i, f), "shape"),
        (lambda: ext.attn_sink_rope_kv_append(q, q, q, c, c2, t, i, f), "k_new"),
        (lambda: ext.attn_sink_rope(q.float(), None, i, f), "bfloat16"),
        (lambda: ext.attn_sink_rope_kv_append(q, q[:, :1], q[:, :1], c, c2, t[:3], i[:3], f), "cu_new"),
        (lambda: ext.attn_sink_rope_kv_append(q, q[:, :1], q[:, :1], c, c2, t, i, f, cu_new=i), "cu_new"),
        (lambda: ext.attn_sink_tree_paged(q, c, c2, t, i, i, i, 1, 1), "cu_seqlens_q"),
        (lambda: ext.attn_sink_tree_paged(q, c, c2, t[:, :0], i, i[:3], i, 1, 1), "page_table"),
        (lambda: ext.attn_sink_tree_paged(q, c, c2[:2], t, i, i, i, 1, 1), "v_cache"),
        (lambda: ext.attn_sink_kv_compact(c, c2, t, i, i), "src"), (lambda: ext.attn_sink_kv_compact(c, c2, t, t, i[:2]), "counts"),
        (lambda: ext.attn_sink_decode_paged_weights(q, c, c2, t, i, w[:2]), "weights"),
        (lambda: ext.attn_sink_evict_paged(c, c2, t, i, w.double(), 4), "weights"),
        (lambda: ext.attn_sink_evict_paged(c, c2, t, i, w, 4, kept=t), "kept"),
    ]
    for call, word in bad:
        with pytest.raises(TypeError, match=word):
            call()
    for call in (lambda: ext.attn_sink_evict_paged(c, c, t, i, w, 4), lambda: ext.attn_sink_evict_paged(c, c2, t, i, w, 0),
                 lambda: ext.attn_sink_kv_compact(c, c, t, t, i), lambda: ext.attn_sink_tree_paged(q, c, c2, t, i.new_zeros(5), i, i, 300, 1)):
        with pytest.raises(ext.AttnSinkError):
            call()
