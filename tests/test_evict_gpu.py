"""Accumulated attention weights, eviction by them, and row moves, against the fp64
definitions.

Tolerances: out and LSE as in test_tree_gpu.py (2^-8 (sum P |v| + |O|) + 2^-13 sum
P |v|; 1.5e-4).  A weight is a sum of probabilities, each off by a factor e^(score
error + LSE error), 3e-4, and the fp32 additions to what was there (2^-23).
Selections and moved rows are exact."""
import numpy as np
import pytest
import torch

from oracle import cache_ops_oracle as co
from cache_ops import paged, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ext():
    from paged_kv_sink_gb300 import build
    build.build()
    import paged_kv_sink_gb300 as ext
    return ext


# ---------------------------------------------------------------------------
# Accumulated weights.


WEIGHTS = [
    # lens, hq, hkv, d, page, first, last, sink
    ([1, 2, 15, 16, 17, 64, 65, 1000], 8, 1, 64, 16, 0, 0, True),
    ([3000, 5, 700], 64, 8, 64, 16, 0, 0, True),
    ([3000, 5, 700], 16, 4, 128, 7, 4, 90, False),
    ([200, 90], 12, 12, 64, 8, 0, 0, False),            # group 1
    ([500, 300], 24, 2, 64, 16, 0, 50, True),           # group 12: two head tiles
    ([130, 300], 40, 2, 128, 32, 0, 0, True),           # group 20: two head blocks
    ([9000], 32, 8, 128, 64, 1024, 7168, False),
    ([0, 7], 8, 2, 64, 16, 0, 0, True),                 # an empty cache
]


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("case", WEIGHTS, ids=lambda c: f"L{max(c[0])}hq{c[1]}-{c[2]}d{c[3]}w{c[5]}-{c[6]}")
def test_weights_match_definition(ext, case, shared):
    lens, hq, hkv, d, page, first, last, sink = case
    k, v, table, sl = paged(lens, hkv, d, page, seed=hq)
    g = torch.Generator().manual_seed(3)
    q = torch.randn(len(lens), hq, d, generator=g).bfloat16()
    sk = torch.rand(hq, generator=g) * 6 - 2 if sink else None
    heads, cap = (1 if shared else hkv), max(lens) + 3
    w0 = torch.rand(len(lens), heads, cap, generator=g)
    dev = [t.cuda() for t in (q, k, v, table, sl)]
    w = w0.clone().cuda()
    out, lse = ext.attn_sink_decode_paged_weights(*dev, w, None if sk is None else sk.cuda(), first, last)
    ref, ref_lse = ext.attn_sink_decode_paged(*dev, None if sk is None else sk.cuda(), first, last)
    torch.cuda.synchronize()
    assert ext.device_status() == 0
    assert same(out, ref) and same(lse, ref_lse)
    w = w.cpu()
    for b, n in enumerate(lens):
        seen = co.in_window(np.arange(n), n - 1, first, last)[None]
        kk, vv = (co.tokens(c, table[b], n) for c in (k, v))
        O, L, P, A = co.attend(q[b:b + 1], kk, vv, seen, None if sk is None else sk.numpy(), d ** -0.5)
        err = np.abs(co.to_np(out[b:b + 1]) - O)
        assert np.all(err <= 2.0 ** -8 * (A + np.abs(O)) + 2.0 ** -13 * A)
        np.testing.assert_allclose(lse[b].cpu().numpy(), L[:, 0], atol=1.5e-4)
        p = P[:, 0].reshape(heads, hq // heads, n).sum(1)
        have, want = w[b, :, :n].numpy(), w0[b, :, :n].numpy() + p
        assert np.all(np.abs(have - want) <= 3e-4 * p + 2.0 ** -23 * want)
        hidden = ~seen[0]
        assert np.array_equal(have[:, hidden], w0[b, :, :n].numpy()[:, hidden])
        assert same(w[b, :, n:], w0[b, :, n:])


def test_weights_accumulate_in_a_fixed_order(ext):
    k, v, table, sl = paged([2500, 40], 2, 64, 16, seed=1)
    g = torch.Generator().manual_seed(4)
    q = torch.randn(2, 16, 64, generator=g).bfloat16().cuda()
    dev = [t.cuda() for t in (k, v, table, sl)]
    runs = []
    for _ in range(2):
        w = torch.zeros(2, 2, 2500, device="cuda")
        for _ in range(3):
            ext.attn_sink_decode_paged_weights(q, *dev, w)
        runs.append(w)
    assert same(*runs)
    # without a sink the weights of a query head sum to 1: 8 heads a KV head, 3 calls
    np.testing.assert_allclose(runs[0].double().sum(-1).cpu().numpy(), 24.0, rtol=3e-4)


def test_weights_with_bad_pages_infinite_sinks_and_a_short_accumulator(ext):
    k, v, table, sl = paged([40, 40], 1, 64, 16, seed=7)
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(5)).bfloat16()
    bad = table.clone()
    bad[1, 1] = 999
    ext.device_status()

    def call(table, w, sink=None):
        ext.attn_sink_decode_paged_weights(q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl.cuda(), w, sink)
        return w.cpu(), ext.device_status()

    w, status = call(bad, torch.zeros(2, 1, 40, device="cuda"))
    assert status == ext._lib.DEV_PAGE_OOB
    assert torch.all(w[1, 0, 16:32] == 0) and torch.all(w[1, 0, :16] > 0)
    np.testing.assert_allclose(w.sum(-1).numpy(), 4.0, rtol=3e-4)
    good, status = call(table, torch.zeros(2, 1, 40, device="cuda"))
    short, status = call(table, torch.zeros(2, 1, 33, device="cuda"))
    assert status == ext._lib.DEV_SEQLEN_OOB and same(short, good[:, :, :33])
    w, status = call(table, torch.zeros(2, 1, 40, device="cuda"), torch.full((4,), float("inf"), device="cuda"))
    assert status == 0 and torch.all(w == 0)
    w, status = call(torch.full_like(table, -5), torch.zeros(2, 1, 40, device="cuda"))  # nothing readable
    assert status == ext._lib.DEV_PAGE_OOB and torch.all(w == 0)


@pytest.mark.parametrize("cap,most", [(5200, 256), (262144, 2240)])
@pytest.mark.parametrize("shared", [True, False])
def test_weights_with_a_table_far_wider_than_the_requests(ext, cap, most, shared):
    """64 requests, most of them short, behind a page table of 262144 tokens: the scratch stays
    below `most` MiB (4 GiB for the table's width: 64 requests, 64 heads, 4 bytes a token), and
    the results are the same as behind a table cut to the longest request."""
    lens = [1 + 37 * b % 450 for b in range(64)]
    lens[20], lens[63] = 5187, 3000
    hkv, hq, heads = 8, 64, 1 if shared else 8
    k, v, table, sl = paged(lens, hkv, 64, 16, seed=41)
    wide = torch.full((64, 262144 // 16), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    g = torch.Generator().manual_seed(42)
    q = torch.randn(64, hq, 64, generator=g).bfloat16()
    dev = [t.cuda() for t in (q, k, v, wide, sl)]
    cut = [*dev[:3], table.cuda(), dev[4]]
    w, w2 = torch.ones(64, heads, cap, device="cuda"), torch.ones(64, heads, cap, device="cuda")
    ref, ref_lse = ext.attn_sink_decode_paged(*dev)
    ext.attn_sink_decode_paged_weights(*(t[:1] if t.shape[0] == 64 else t for t in cut), w2[:1].clone())
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    out, lse = ext.attn_sink_decode_paged_weights(*dev, w)
    torch.cuda.synchronize()
    assert free - torch.cuda.mem_get_info()[0] <= most << 20
    assert ext.device_status() == 0
    assert same(out, ref) and same(lse, ref_lse)
    ext.attn_sink_decode_paged_weights(*cut, w2)
    # each weight is off by a factor of at most 3e-4, and one fp32 addition to 1
    p, p2 = w.double() - 1.0, w2.double() - 1.0
    assert torch.all((p - p2).abs() <= 6e-4 * p.abs() + 2.0 ** -22)
    for b in (0, 20, 63):
        n = lens[b]
        kk, vv = (co.tokens(c, table[b], n) for c in (k, v))
        _, _, P, _ = co.attend(q[b:b + 1], kk, vv, np.ones((1, n), bool), None, 0.125)
        want = P[:, 0].reshape(heads, hq // heads, n).sum(1)
        have = w[b].cpu().double().numpy()
        assert np.all(np.abs(have[:, :n] - 1.0 - want) <= 3e-4 * want + 2.0 ** -23 * (1.0 + want))
        assert np.all(have[:, n:] == 1.0)


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("hq,hkv", [(3, 3), (6, 3), (9, 3), (12, 3), (5, 1), (12, 2), (7, 1), (8, 1), (9, 1), (32, 2), (34, 2)])
def test_weights_of_every_group_size(ext, hq, hkv, shared):
    """1 to 8 query heads a KV head, one tile of heads, and more."""
    lens = [130, 1, 700]
    k, v, table, sl = paged(lens, hkv, 64, 16, seed=hq)
    q = torch.randn(3, hq, 64, generator=torch.Generator().manual_seed(45)).bfloat16()
    heads = 1 if shared else hkv
    dev = [t.cuda() for t in (q, k, v, table, sl)]
    w = torch.zeros(3, heads, 701, device="cuda")
    out, lse = ext.attn_sink_decode_paged_weights(*dev, w)
    ref, ref_lse = ext.attn_sink_decode_paged(*dev)
    assert ext.device_status() == 0 and same(out, ref) and same(lse, ref_lse)
    for b, n in enumerate(lens):
        kk, vv = (co.tokens(c, table[b], n) for c in (k, v))
        _, _, P, _ = co.attend(q[b:b + 1], kk, vv, np.ones((1, n), bool), None, 0.125)
        want = P[:, 0].reshape(heads, hq // heads, n).sum(1)
        assert np.all(np.abs(w[b, :, :n].cpu().numpy() - want) <= 3e-4 * want) and not w[b, :, n:].any()


def test_scores_take_no_more_room_than_the_heads_need(ext):
    """64 requests, 8 query heads over 8 KV heads, accumulators of 65536 tokens: 134 MB of scores."""
    lens = [40] * 64
    k, v, table, sl = paged(lens, 8, 64, 16, seed=46)
    wide = torch.full((64, 4096), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    dev = [t.cuda() for t in (torch.ones(64, 8, 64).bfloat16(), k, v, wide, sl)]
    w = torch.zeros(64, 8, 65536, device="cuda")
    ext.attn_sink_decode_paged(*dev)
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    ext.attn_sink_decode_paged_weights(*dev, w)
    torch.cuda.synchronize()
    assert free - torch.cuda.mem_get_info()[0] <= 256 << 20
    np.testing.assert_allclose(w.sum(-1).cpu().numpy(), 1.0, rtol=3e-4)


@pytest.mark.parametrize("first,last", [(0, 0), (10, 50)])
def test_weights_with_a_bound_of_the_lengths(ext, first, last):
    """With max_seqlen the call behind a wide table is the one behind a table cut there, bit for
    bit; a request past the bound is cut there and reported."""
    lens, bound = [5000, 3, 640, 4096], 4096
    k, v, table, sl = paged(lens, 2, 64, 16, seed=43)
    wide = torch.full((4, 8192), -1, dtype=torch.int32)
    wide[:, :table.shape[1]] = table
    q = torch.randn(4, 16, 64, generator=torch.Generator().manual_seed(44)).bfloat16()
    sink = torch.zeros(16, device="cuda")
    got = []
    ext.device_status()
    for t, n, kw in ((wide, sl, dict(max_seqlen=bound)), (table[:, :bound // 16].contiguous(), sl.clamp(max=bound), {})):
        w = torch.zeros(4, 2, 8192 * 16, device="cuda")
        got.append((*ext.attn_sink_decode_paged_weights(q.cuda(), k.cuda(), v.cuda(), t.cuda(), n.cuda(), w, sink, first,
                                                        last, **kw), w))
        assert ext.device_status() == (ext._lib.DEV_SEQLEN_OOB if kw else 0)
    for a, b in zip(*got):
        assert same(a, b)
    dev = [t.cuda() for t in (q, k, v, wide, sl)]
    a, b = (ext.attn_sink_decode_paged_weights(*dev, w.clone(), **kw) for kw in ({}, dict(max_seqlen=2 ** 32 + 7)))
    assert same(a[0], b[0]) and same(a[1], b[1]) and ext.device_status() == 0
    got = [ext.attn_sink_decode_paged_weights(q.cuda(), k.cuda(), v.cuda(), wide.cuda(), sl.cuda(), w, max_seqlen=0)]
    assert torch.all(got[0][0] == 0) and torch.all(torch.isneginf(got[0][1]))
    assert ext.device_status() == ext._lib.DEV_SEQLEN_OOB


@pytest.mark.parametrize("hq,hkv", [(2, 2), (6, 2), (24, 2)])
@pytest.mark.parametrize("shared", [False, True])
def test_weights_of_infinite_keys(ext, hq, hkv, shared):
    # token 5's scores are -inf for every head: its weight is 0, and the others sum to 1 per head
    k, v, table, sl = paged([40], hkv, 64, 16, seed=8)
    q = torch.rand(1, hq, 64, generator=torch.Generator().manual_seed(6)).bfloat16() + 0.5
    k.view(-1, hkv, 64)[co.slot(table[0].numpy(), 16, np.array([5]))] = float("-inf")
    w = torch.zeros(1, 1 if shared else hkv, 40, device="cuda")
    ext.attn_sink_decode_paged_weights(q.cuda(), k.cuda(), v.cuda(), table.cuda(), sl.cuda(), w)
    w = w.cpu()
    assert ext.device_status() == 0 and torch.all(w[:, :, 5] == 0)
    np.testing.assert_allclose(w.sum(-1).numpy(), hq / w.shape[1], rtol=3e-4)


# ---------------------------------------------------------------------------
# Eviction.


def evict_reference(k, v, table, lens, w, budget, first, last):
    """Moved caches, kept lists and weights by the definition (whole heads)."""
    k, v = k.clone(), v.clone()
    B, heads, cap = w.shape
    hkv, page = k.shape[2], k.shape[1]
    kept = torch.full((B, heads, budget), -1, dtype=torch.int32)
    w_out = torch.zeros_like(w)
    for b, n in enumerate(lens):
        for h in range(heads):
            src = co.evict(w[b, h].numpy(), n, budget, first, last)
            kept[b, h, :len(src)] = torch.from_numpy(src).int()
            w_out[b, h, :len(src)] = w[b, h, torch.from_numpy(src)]
            a = torch.from_numpy(co.slot(table[b].numpy(), page, src))
            z = torch.from_numpy(co.slot(table[b].numpy(), page, np.arange(len(src))))
            per = slice(h, h + 1) if heads == hkv else slice(None)
            for c in (k, v):
                rows = c.view(-1, hkv, c.shape[3])
                rows[z, per] = rows[a, per]
    return k, v, kept, w_out


EVICT = [
    # lens, hkv, d, page, budget, first, last, kind
    ([100, 64, 65, 1, 0, 63], 2, 64, 16, 64, 4, 16, "random"),
    ([5000, 300, 2049], 3, 128, 64, 1024, 4, 200, "random"),
    ([5000, 2000], 2, 64, 7, 1500, 0, 0, "ties"),           # most weights equal; odd pages
    ([900, 800], 4, 64, 8, 256, 100, 156, "random"),        # nothing free: the protected alone
    ([700], 1, 64, 16, 1, 0, 0, "random"),                  # one token stays
    ([700], 1, 64, 16, 1, 0, 1, "random"),
    ([1200, 1100], 12, 64, 16, 1000, 0, 1, "zeros"),
    ([600, 512], 2, 128, 16, 300, 10, 20, "odd"),           # NaN, infinities, negative, -0, subnormal
    ([33000], 2, 64, 128, 20000, 4, 64, "small range"),     # equal leading digits of the key
]


def weight_values(kind, shape, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(*shape, generator=g) ** 4
    if kind == "ties":
        w = (w * 3).round()
    elif kind == "zeros":
        w = torch.zeros(shape)
    elif kind == "odd":
        odd = torch.tensor([float("nan"), float("inf"), float("-inf"), -1.0, -0.0, 0.0, 1e-41, -1e-41, 2.0])
        w = odd[torch.randint(0, len(odd), shape, generator=g)]
    elif kind == "small range":
        w = 1.0 + w * 2.0 ** -14
    return w


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("case", EVICT, ids=lambda c: f"L{max(c[0])}h{c[1]}d{c[2]}ps{c[3]}b{c[4]}-{c[5]}-{c[6]}{c[7]}")
def test_evict_matches_definition(ext, case, shared, in_place):
    lens, hkv, d, page, budget, first, last, kind = case
    k, v, table, sl = paged(lens, hkv, d, page, seed=budget)
    w = weight_values(kind, (len(lens), 1 if shared else hkv, max(lens) + 5), seed=2)
    want_k, want_v, want_kept, want_w = evict_reference(k, v, table, lens, w, budget, first, last)
    kc, vc, wc = k.cuda(), v.cuda(), w.cuda()
    out = None if in_place else torch.full_like(wc, 5.0)
    new, kept = ext.attn_sink_evict_paged(kc, vc, table.cuda(), sl.cuda(), wc, budget, first, last, weights_out=out)
    torch.cuda.synchronize()
    assert ext.device_status() == 0
    assert torch.equal(new.cpu(), sl.clamp(max=budget)) and torch.equal(kept.cpu(), want_kept)
    assert same((wc if in_place else out).cpu(), want_w)
    if not in_place:
        assert same(wc.cpu(), w)
    for b, n in enumerate(lens):   # what is kept; the freed slots hold anything
        rows = torch.from_numpy(co.slot(table[b].numpy(), page, np.arange(min(n, budget))))
        for got, want in ((kc, want_k), (vc, want_v)):
            assert same(got.cpu().view(-1, hkv, d)[rows], want.view(-1, hkv, d)[rows])


@pytest.mark.parametrize("lens,budget,kind", [
    ([200000, 150000], 70000, "random"),          # two rounds of keys in each CTA of a cluster
    ([40000] + [50] * 79, 18000, "ties"),         # three rounds in one CTA
    ([131073], 131072, "ties"), ([131073], 1, "random")])
def test_evict_long_lists(ext, lens, budget, kind):
    k, v, table, sl = paged(lens, 1, 64, 64, seed=budget)
    first, last = (4, 1000) if budget > 1 else (0, 0)
    w = weight_values(kind, (len(lens), 1, max(lens)), seed=2)
    want_k, want_v, want_kept, want_w = evict_reference(k, v, table, lens, w, budget, first, last)
    kc, vc, wc = k.cuda(), v.cuda(), w.cuda()
    new, kept = ext.attn_sink_evict_paged(kc, vc, table.cuda(), sl.cuda(), wc, budget, first, last)
    assert ext.device_status() == 0
    assert torch.equal(new.cpu(), sl.clamp(max=budget)) and torch.equal(kept.cpu(), want_kept)
    assert same(wc.cpu(), want_w)
    kc, vc = kc.cpu(), vc.cpu()
    for b, n in enumerate(lens):
        rows = torch.from_numpy(co.slot(table[b].numpy(), 64, np.arange(min(n, budget))))
        assert same(kc.view(-1, 64)[rows], want_k.view(-1, 64)[rows])
        assert same(vc.view(-1, 64)[rows], want_v.view(-1, 64)[rows])


def test_evict_refuses_nothing_it_documents(ext):
    """Lengths past the accumulator or the page table are cut there, with a status bit;
    pages of other requests stay as they were."""
    k, v, table, sl = paged([100, 100], 2, 64, 16, seed=3)
    w = torch.rand(2, 2, 60, generator=torch.Generator().manual_seed(1))
    kc, vc = k.cuda(), v.cuda()
    ext.device_status()
    new, kept = ext.attn_sink_evict_paged(kc, vc, table.cuda(), torch.tensor([100, 30]).int().cuda(), w.cuda(), 40)
    assert ext.device_status() == ext._lib.DEV_SEQLEN_OOB
    assert new.tolist() == [40, 30]
    assert kept[0, 1].tolist() == co.evict(w[0, 1].numpy(), 60, 40, 0, 0).tolist()
    pages = table[1, :7].long()
    assert same(kc.cpu()[pages], k[pages]) and same(vc.cpu()[pages], v[pages])


def test_decode_after_eviction_equals_decode_over_the_kept(ext):
    k, v, table, sl = paged([900, 700, 20], 2, 64, 16, seed=4)
    g = torch.Generator().manual_seed(6)
    q = torch.randn(3, 8, 64, generator=g).bfloat16()
    kc, vc, tc, sc = k.cuda(), v.cuda(), table.cuda(), sl.cuda()
    w = torch.zeros(3, 2, 900, device="cuda")
    for s in range(3):
        ext.attn_sink_decode_paged_weights(torch.roll(q, s, 1).cuda(), kc, vc, tc, sc, w)
    w_before = w.cpu().clone()
    new, kept = ext.attn_sink_evict_paged(kc, vc, tc, sc, w, 128, keep_first=4, keep_last=32)
    out, lse = ext.attn_sink_decode_paged(q.cuda(), kc, vc, tc, new)
    torch.cuda.synchronize()
    for b, n in enumerate([900, 700, 20]):
        for h in range(2):
            src = co.evict(w_before[b, h].numpy(), n, 128, 4, 32)
            kk, vv = (co.tokens(c, table[b], n)[src][:, h:h + 1] for c in (k, v))
            O, L, _, A = co.attend(q[b:b + 1, 4 * h:4 * h + 4], kk, vv, np.ones((1, len(src)), bool), None, 0.125)
            err = np.abs(co.to_np(out[b:b + 1, 4 * h:4 * h + 4]) - O)
            assert np.all(err <= 2.0 ** -8 * (A + np.abs(O)) + 2.0 ** -13 * A)
            np.testing.assert_allclose(lse[b, 4 * h:4 * h + 4].cpu().numpy(), L[:, 0], atol=1.5e-4)


# ---------------------------------------------------------------------------
# Row moves.


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("hkv,d,page,most", [(2, 64, 16, 9), (3, 128, 8, 200), (1, 64, 5, 1), (12, 64, 64, 3000)])
def test_compact_moves_rows(ext, hkv, d, page, most, per_head):
    g = torch.Generator().manual_seed(most)
    lens = [most * 2 + 40, most + 7, most + 1]
    k, v, table, sl = paged(lens, hkv, d, page, seed=most)
    base = torch.tensor([17, 3, 0]).int()
    counts = torch.tensor([most, most // 2, 0]).int()
    heads = hkv if per_head else 1
    src = torch.zeros(3, heads, most, dtype=torch.int32)
    for b in range(3):
        for h in range(heads):
            n = int(counts[b])
            span = lens[b] - int(base[b])
            src[b, h, :n] = int(base[b]) + torch.randperm(span, generator=g)[:n].sort().values.int()
    want = [k.clone(), v.clone()]
    for b in range(3):
        for h in range(heads):
            n = int(counts[b])
            a = torch.from_numpy(co.slot(table[b].numpy(), page, src[b, h, :n].numpy()))
            z = torch.from_numpy(co.slot(table[b].numpy(), page, int(base[b]) + np.arange(n)))
            per = slice(h, h + 1) if per_head else slice(None)
            for c in want:
                rows = c.view(-1, hkv, d)
                rows[z, per] = rows[a, per]
    kc, vc = k.cuda(), v.cuda()
    ext.attn_sink_kv_compact(kc, vc, table.cuda(), (src if per_head else src[:, 0]).contiguous().cuda(),
                             counts.cuda(), base.cuda())
    torch.cuda.synchronize()
    assert ext.device_status() == 0
    assert same(kc.cpu(), want[0]) and same(vc.cpu(), want[1])   # all slots, the untouched ones too


def test_compact_skips_rows_out_of_order(ext):
    k, v, table, sl = paged([64, 64], 2, 64, 16, seed=11)
    ext.device_status()

    def call(src, counts, base=None):
        kc, vc = k.cuda(), v.cuda()
        ext.attn_sink_kv_compact(kc, vc, table.cuda(), torch.tensor(src).int().cuda(), torch.tensor(counts).int().cuda(),
                                 None if base is None else torch.tensor(base).int().cuda())
        return kc.cpu(), ext.device_status()

    kc, status = call([[5, 5, 9], [1, 2, 3]], [3, 3])           # the same token twice
    assert status == ext._lib.DEV_ORDER
    one = co.slot(table[1].numpy(), 16, np.arange(4))
    assert same(kc.view(-1, 2, 64)[one[:3]], k.view(-1, 2, 64)[one[1:]])
    kc, status = call([[5, 6, 9], [1, 2, 3]], [3, 3], [7, 0])   # before its destination
    assert status == ext._lib.DEV_ORDER
    kc, status = call([[5, 6, 900], [1, 2, 3]], [3, 3])         # past the page table
    assert status == ext._lib.DEV_SEQLEN_OOB
    kc, status = call([[5, 6, 9], [1, 2, 3]], [9, -1])          # more rows than the list, fewer than none
    assert status == ext._lib.DEV_SEQLEN_OOB
    assert same(kc.view(-1, 2, 64)[one], k.view(-1, 2, 64)[one])


def test_compact_refuses_destinations_past_the_page_table(ext):
    k, v, table, sl = paged([64], 2, 64, 16, seed=12)
    tokens = table.shape[1] * 16
    src = torch.tensor([[1, 2, 3, 4]]).int().cuda()
    ext.device_status()
    for base in (tokens, 2 ** 31 - 3, 2 ** 31 - 1, -1):
        kc, vc = k.cuda(), v.cuda()
        ext.attn_sink_kv_compact(kc, vc, table.cuda(), src, torch.tensor([4]).int().cuda(), torch.tensor([base]).int().cuda())
        assert ext.device_status() == ext._lib.DEV_SEQLEN_OOB
        assert same(kc.cpu(), k) and same(vc.cpu(), v)


def test_evict_and_weights_in_a_graph(ext):
    """A captured decode-and-evict step, replayed on new contents, equals the eager one."""
    k, v, table, sl = paged([300, 200], 2, 64, 16, seed=12)
    q = torch.randn(2, 8, 64, generator=torch.Generator().manual_seed(7)).bfloat16().cuda()
    tc, sc = table.cuda(), sl.cuda()
    kc, vc, w = k.cuda(), v.cuda(), torch.zeros(2, 2, 300, device="cuda")
    new, kept = torch.empty_like(sc), torch.empty(2, 2, 64, dtype=torch.int32, device="cuda")

    def step():
        out, _ = ext.attn_sink_decode_paged_weights(q, kc, vc, tc, sc, w)
        ext.attn_sink_evict_paged(kc, vc, tc, sc, w, 64, 2, 8, kept=kept, new_seqlens=new)
        return out

    def reset():
        kc.copy_(k), vc.copy_(v), w.zero_()

    out = step()
    want = [x.clone() for x in (out, kept, new, w)]
    want_rows = kc.clone()
    reset()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    reset()
    for _ in range(2):
        reset()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip((out, kept, new, w), want):
            assert torch.equal(a, b)
        for b in range(2):
            rows = torch.from_numpy(co.slot(table[b].numpy(), 16, np.arange(64))).cuda()
            assert same(kc.view(-1, 2, 64)[rows], want_rows.view(-1, 2, 64)[rows])
