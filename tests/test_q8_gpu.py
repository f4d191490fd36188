"""The 8-bit paged cache: codes and scales against the definition bit for bit, attention over
it against fp64.

Tolerances.  With A = sum P |v| and S = max_t scale sum |q_i k_ti|:
 * a score is off by d + 8 fp32 roundings of terms that sum to at most S (products' sums,
   scales, the factor log2 e and its place in the exponent), so by delta = (d + 8) 2^-24 S;
   every weight and the denominator by e^delta each;
 * weights meet V in fp16 (2^-11 of each) or, where tokens are expanded, bf16 (2^-8);
   the exponentials are off by at most 2^-21;
 * O is rounded to bf16: 2^-8 |O|.
Together |err| <= 2^-8 |O| + (w + 2 delta + 2^-20) A with w 2^-11 or 2^-8, and for the lse
delta + 2^-20 (1 + |lse|)."""
import numpy as np
import pytest
import torch

from oracle import cache_ops_oracle as co
from oracle import serving_oracle as so
from cache_ops import cu, same

pytestmark = pytest.mark.gpu
FMT = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


@pytest.fixture(scope="module")
def ext():
    from paged_kv_sink_gb300 import build
    build.build()
    import paged_kv_sink_gb300 as ext
    return ext


def table_for(lens, page, g, extra=2, spare=1):
    n = [-(-t // page) for t in lens]
    perm = torch.randperm(sum(n) + extra, generator=g).int()
    table = torch.full((len(lens), max(n + [0]) + spare), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(n):
        table[b, :m] = perm[at:at + m]
        at += m
    return table, sum(n) + extra


class Cache:
    """An 8-bit cache with random codes in its requests' tokens and NaN-like ones elsewhere (0x7f: e4m3
    NaN, int8 127), scales of several sizes (`any_scale`: not powers of two)."""

    def __init__(self, lens, hkv, d, page, block, fmt, seed=0, any_scale=False, spread=2.0):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.page, self.block, self.lens = fmt, page, block, list(lens)
        self.table, pool = table_for(lens, page, g)
        self.codes, self.scales = [], []
        for _ in range(2):
            x = torch.randint(0, 256, (pool, page, hkv, d), generator=g).to(torch.uint8)
            x = torch.where((x & 127) == 127, x - 1, x) if fmt == "e4m3" else torch.where(x == 128, 129, x).to(torch.uint8)
            own = torch.zeros(pool, page, dtype=torch.bool)
            for b, n in enumerate(lens):
                for t in range(n):
                    own[self.table[b, t // page], t % page] = True
            x[~own] = 127
            s = torch.exp2(torch.round((torch.rand(pool, page // block, hkv, generator=g) * 2 - 1) * spread))
            s *= 2.0 ** (-8 if fmt == "e4m3" else -6)
            if any_scale:
                s *= 0.5 + torch.rand(s.shape, generator=g)
            self.codes.append(x)
            self.scales.append(s.float())

    def dev(self):
        return [c.view(FMT[self.fmt]).cuda() for c in self.codes] + [s.cuda() for s in self.scales] + [self.table.cuda()]

    def tokens(self, b):
        out = []
        for c, s in zip(self.codes, self.scales):
            full = so.expand(c.numpy(), s.numpy(), self.fmt)
            n = self.lens[b]
            t = np.arange(n)
            out.append(full[self.table[b].numpy()[t // self.page], t % self.page])
        return out


def check(out, lse, q, k, v, seen, sink, w, scale=None):
    """out (n, hq, d), lse (hq, n) of one request."""
    n, hq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    O, L, P, A = co.attend(q, k, v, seen, sink, scale)
    S = scale * np.abs(co.to_np(q)).reshape(n, hq, d).max(initial=0) * np.abs(k).sum(-1).max(initial=0)
    delta = (d + 8) * 2.0 ** -24 * S
    err = np.abs(co.to_np(out) - O)
    assert np.all(err <= 2.0 ** -8 * np.abs(O) + (w + 2 * delta + 2.0 ** -20) * A), (err.max(), A.max())
    got = co.to_np(lse)
    fine = np.isfinite(L)
    assert np.array_equal(got[~fine], L[~fine])
    assert np.all(np.abs(got[fine] - L[fine]) <= delta + 2.0 ** -20 * (1 + np.abs(L[fine])))


# ---------------------------------------------------------------------------
# Append.

APPEND = [
    # prefix lengths, new rows, hkv, d, page, block
    ([0, 1, 15, 16, 17, 300], [1, 1, 1, 1, 1, 1], 8, 64, 16, 16),
    ([0, 5, 40, 7], [70, 1, 0, 3], 2, 64, 16, 8),
    ([0, 33, 2], [200, 31, 130], 3, 128, 64, 32),
    ([3, 0], [40, 22], 1, 128, 7, 7),
    ([10, 0, 9], [5, 61, 1], 2, 64, 24, 8),
    ([100, 0], [300, 257], 1, 64, 128, 128),
    ([1, 6], [9, 4], 2, 128, 8, 1),
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"n{max(c[1])}h{c[2]}d{c[3]}p{c[4]}b{c[5]}")
def test_append_codes_and_scales_are_exact(ext, case, fmt):
    prefix, new, hkv, d, page, block = case
    total = [p + n for p, n in zip(prefix, new)]
    c = Cache(total, hkv, d, page, block, fmt, seed=d + page)
    g = torch.Generator().manual_seed(9)
    rows = [(torch.randn(sum(new), hkv, d, generator=g) * torch.exp2(torch.randint(-12, 12, (sum(new), hkv, 1), generator=g).float())
             * 2.0 ** -7).bfloat16() for _ in range(2)]
    want = [(x.numpy().copy(), s.numpy().astype(np.float64)) for x, s in zip(c.codes, c.scales)]
    at = 0
    for b, n in enumerate(new):
        for (x, s), r in zip(want, rows):
            if n:
                so.append(x, s, co.to_np(r[at:at + n]), c.table[b].numpy(), total[b], block, fmt)
        at += n
    dev = c.dev()
    sl = torch.tensor(total, dtype=torch.int32).cuda()
    got = ext.attn_sink_kv_append_q8(*[r.cuda() for r in rows], *dev, sl, cu_new=cu(new).cuda())
    assert ext.device_status() == 0
    for i in range(2):
        np.testing.assert_array_equal(got[2 + i].cpu().double().numpy(), want[i][1])
        np.testing.assert_array_equal(so.values(got[i].cpu().view(torch.uint8).numpy(), fmt), so.values(want[i][0], fmt))
        assert got[i] is dev[i]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_of_strided_rows_token_by_token(ext, fmt):
    """Columns of a packed buffer, one token a call without cu_new, blocks that grow."""
    page, block, hkv, d = 16, 8, 2, 64
    c = Cache([20, 20], hkv, d, page, block, fmt, seed=3)
    g = torch.Generator().manual_seed(4)
    dev = c.dev()
    want = [(x.numpy().copy(), s.numpy().astype(np.float64)) for x, s in zip(c.codes, c.scales)]
    for t in range(20):
        packed = (torch.randn(2, 6, d, generator=g) * 2.0 ** (t - 10)).bfloat16()
        k, v = packed.cuda()[:, 2:4], packed.cuda()[:, 4:6]
        sl = torch.full((2,), t + 1, dtype=torch.int32).cuda()
        ext.attn_sink_kv_append_q8(k, v, *dev, sl)
        for b in range(2):
            for i, r in enumerate((packed[:, 2:4], packed[:, 4:6])):
                so.append(*want[i], co.to_np(r[b:b + 1]), c.table[b].numpy(), t + 1, block, fmt)
    for i in range(2):
        np.testing.assert_array_equal(dev[2 + i].cpu().double().numpy(), want[i][1])
        np.testing.assert_array_equal(so.values(dev[i].cpu().view(torch.uint8).numpy(), fmt), so.values(want[i][0], fmt))
    assert ext.device_status() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_of_values_that_are_not_numbers(ext, fmt):
    c = Cache([8, 8, 8, 8], 1, 64, 8, 8, fmt)
    x = torch.randn(32, 1, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    x[3, 0, 5], x[9, 0, 0], x[10, 0, 63] = float("inf"), float("nan"), float("-inf")
    x[16:24] = float("nan")
    x[24:] = 0
    want = [(a.numpy().copy(), s.numpy().astype(np.float64)) for a, s in zip(c.codes, c.scales)]
    for b in range(4):
        for a in want:
            so.append(*a, co.to_np(x[8 * b:8 * b + 8]), c.table[b].numpy(), 8, 8, fmt)
    dev = c.dev()
    ext.attn_sink_kv_append_q8(x.cuda(), x.cuda(), *dev, torch.full((4,), 8).int().cuda(), cu_new=cu([8] * 4).cuda(), max_new=8)
    assert ext.device_status() == ext._lib.DEV_VALUE
    for i in range(2):
        np.testing.assert_array_equal(dev[2 + i].cpu().double().numpy(), want[i][1])
        np.testing.assert_array_equal(so.values(dev[i].cpu().view(torch.uint8).numpy(), fmt), so.values(want[i][0], fmt))
    assert dev[2].min() >= 2.0 ** -64


def test_append_skips_what_is_out_of_range(ext):
    """A bad page, rows past max_new, rows past the tensor, a table that is too short, fewer tokens
    than rows: reported, and nothing else is written."""
    D = ext._lib
    def run(edit, new, total, rows=None, max_new=None):
        c = Cache([40, 40], 1, 64, 8, 8, "int8", seed=8)
        edit(c)
        dev = c.dev()
        x = torch.ones(sum(new) if rows is None else rows, 1, 64).bfloat16().cuda()
        ext.device_status()
        ext.attn_sink_kv_append_q8(x, x, *dev, torch.tensor(total).int().cuda(), cu_new=cu(new).cuda(),
                                   max_new=max(new) if max_new is None else max_new)
        changed = (dev[0].cpu().view(torch.uint8) != c.codes[0]).any(-1).any(-1)
        where = {(b, t) for b in range(2) for t in range(40)
                 if 0 <= c.table[b, t // 8] < 11 and changed[c.table[b, t // 8], t % 8]}
        return where, ext.device_status()

    def bad(c):
        c.table[0, 1] = 999
    span = lambda b, lo, hi: {(b, t) for t in range(lo, hi)}
    where, st = run(bad, [24, 0], [24, 40])
    assert st == D.DEV_PAGE_OOB and where == span(0, 0, 8) | span(0, 16, 24)
    where, st = run(lambda c: None, [20, 3], [20, 10], max_new=16)
    assert st == D.DEV_SEQLEN_OOB and where == span(0, 0, 16) | span(1, 7, 10)
    where, st = run(lambda c: None, [16, 16], [16, 16], rows=24)
    assert st == D.DEV_SEQLEN_OOB and where == span(0, 0, 16) | span(1, 0, 8)
    where, st = run(lambda c: None, [60, 0], [60, 8])
    assert st == D.DEV_SEQLEN_OOB | D.DEV_PAGE_OOB and where == span(0, 0, 40)  # 48 slots of table, the last page -1
    where, st = run(lambda c: None, [12, 0], [8, 8])
    assert st == D.DEV_SEQLEN_OOB and where == span(0, 0, 8)


# ---------------------------------------------------------------------------
# Decode.

DECODE = [
    # lens, hq, hkv, d, page, block, first, last, sink
    ([1, 2, 31, 32, 33, 127, 128, 129, 1000], 8, 1, 64, 16, 16, 0, 0, True),
    ([3000, 5, 700], 64, 8, 64, 16, 16, 0, 0, True),
    ([3000, 5, 700], 16, 4, 128, 7, 7, 4, 90, False),
    ([200, 90], 12, 12, 64, 8, 4, 0, 0, False),             # group 1
    ([500, 300], 24, 2, 64, 24, 8, 0, 50, True),            # group 12
    ([130, 300], 40, 2, 128, 32, 32, 0, 0, True),           # group 20: two row tiles
    ([130, 300], 40, 2, 64, 32, 1, 3, 40, True),            # group 20: one
    ([77, 513], 80, 1, 64, 128, 64, 0, 0, False),           # group 80: three
    ([9000], 32, 8, 128, 64, 64, 1024, 7168, False),
    ([0, 7], 8, 2, 64, 16, 16, 0, 0, True),                 # an empty cache
    ([0, 7], 8, 2, 128, 16, 16, 0, 0, False),
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("case", DECODE, ids=lambda c: f"L{max(c[0])}hq{c[1]}-{c[2]}d{c[3]}p{c[4]}w{c[6]}-{c[7]}")
def test_decode_matches_definition(ext, case, fmt):
    lens, hq, hkv, d, page, block, first, last, sink = case
    c = Cache(lens, hkv, d, page, block, fmt, seed=hq, any_scale=hq == 16)
    g = torch.Generator().manual_seed(3)
    q = torch.randn(len(lens), hq, d, generator=g).bfloat16()
    sk = torch.rand(hq, generator=g) * 6 - 2 if sink else None
    dev = c.dev()
    sl = torch.tensor(lens).int().cuda()
    out, lse = ext.attn_sink_decode_paged_q8(q.cuda(), *dev, sl, None if sk is None else sk.cuda(), first, last)
    bounded, lse2 = ext.attn_sink_decode_paged_q8(q.cuda(), *dev, sl, None if sk is None else sk.cuda(), first, last,
                                                  max_seqlen=max(lens))
    assert ext.device_status() == 0
    for b, n in enumerate(lens):
        k, v = c.tokens(b)
        seen = so.chunk_seen(n, 1, first, last) if n else np.zeros((1, 0), bool)
        for o, z in ((out, lse), (bounded, lse2)):
            check(o[b:b + 1].cpu(), z[b][:, None].cpu(), q[b:b + 1], k, v, seen, None if sk is None else sk.numpy(), 2.0 ** -11)


def test_decode_with_scales_far_apart(ext):
    """V's scales differ by 2^60 between blocks, K's by 2^20: the weights stay in fp16's range."""
    c = Cache([400, 400], 2, 64, 16, 8, "e4m3", seed=5)
    g = torch.Generator().manual_seed(5)
    c.scales[0] = torch.exp2(torch.randint(-24, -4, c.scales[0].shape, generator=g).float())
    c.scales[1] = torch.exp2(torch.randint(-30, 30, c.scales[1].shape, generator=g).float())
    c.scales[1][:, 0] = 2.0 ** 30  # some of the largest everywhere
    q = torch.randn(2, 8, 64, generator=g).bfloat16()
    out, lse = ext.attn_sink_decode_paged_q8(q.cuda(), *c.dev(), torch.tensor([400, 400]).int().cuda())
    for b in range(2):
        k, v = c.tokens(b)
        check(out[b:b + 1].cpu(), lse[b][:, None].cpu(), q[b:b + 1], k, v, np.ones((1, 400), bool), None, 2.0 ** -11)


@pytest.mark.parametrize("big", [1e-30, 1e4, 1e30])
def test_decode_with_queries_of_any_size(ext, big):
    """q leaves fp16's range; a scale brings the scores back."""
    c = Cache([300], 1, 128, 16, 16, "int8", seed=6)
    q = (torch.randn(1, 4, 128, generator=torch.Generator().manual_seed(6)) * big).bfloat16()
    out, lse = ext.attn_sink_decode_paged_q8(q.cuda(), *c.dev(), torch.tensor([300]).int().cuda(), scale=0.1 / big)
    k, v = c.tokens(0)
    check(out.cpu(), lse.t().cpu(), q, k, v, np.ones((1, 300), bool), None, 2.0 ** -11, scale=float(np.float32(0.1 / big)))


def test_many_equal_tokens_keep_their_weight(ext):
    """200k tokens with nearly the same weight, far below one token's: sums do not lose them."""
    n, page = 200000, 128
    c = Cache([n], 1, 64, page, 128, "int8", seed=7, spread=0)
    q = torch.zeros(1, 1, 64)
    q[0, 0, 0] = 1.0
    codes = c.codes[0].view(torch.int8)
    codes[:, :, :, 0] = 0
    codes[c.table[0, 3], 5, 0, 0] = 127
    c.scales[0][:] = 1.0
    c.codes[1].view(torch.int8)[:] = 64
    c.codes[1].view(torch.int8)[c.table[0, 3], 5] = -64
    out, lse = ext.attn_sink_decode_paged_q8(q.bfloat16().cuda(), *c.dev(), torch.tensor([n]).int().cuda(), scale=0.1)
    k, v = c.tokens(0)
    check(out.cpu(), lse.t().cpu(), q, k, v, np.ones((1, n), bool), None, 2.0 ** -11, scale=float(np.float32(0.1)))
    # the rest's weights are e^-12.7 of that token's, their sum 0.61 of it: 1 (0.61 - 1) / 1.61
    assert -0.26 < float(out[0, 0, 0]) < -0.22


def test_decode_reports_bad_pages_and_lengths(ext):
    c = Cache([64, 64, 64], 1, 64, 16, 16, "e4m3", seed=9)
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(9)).bfloat16()
    c.table = c.table[:, :4].contiguous()
    c.table[1, 2] = -7
    ext.device_status()
    out, lse = ext.attn_sink_decode_paged_q8(q.cuda(), *c.dev(), torch.tensor([64, 64, 65]).int().cuda())
    assert ext.device_status() == ext._lib.DEV_PAGE_OOB | ext._lib.DEV_SEQLEN_OOB
    c.table[1, 2] = 0
    for b in range(3):
        k, v = c.tokens(b)
        seen = np.ones((1, 64), bool)
        if b == 1:
            seen[0, 32:48] = False  # takes no weight
        check(out[b:b + 1].cpu(), lse[b][:, None].cpu(), q[b:b + 1], k, v, seen, None, 2.0 ** -11)


@pytest.mark.parametrize("sink", [float("inf"), float("-inf"), 80.0])
def test_decode_sinks_at_their_ends(ext, sink):
    c = Cache([50, 0], 1, 64, 16, 16, "e4m3", seed=2)
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(2)).bfloat16()
    out, lse = ext.attn_sink_decode_paged_q8(q.cuda(), *c.dev(), torch.tensor([50, 0]).int().cuda(), torch.full((4,), sink).cuda())
    for b, n in enumerate((50, 0)):
        k, v = c.tokens(b)
        check(out[b:b + 1].cpu(), lse[b][:, None].cpu(), q[b:b + 1], k, v, np.ones((1, n), bool), np.full(4, sink), 2.0 ** -11)


# ---------------------------------------------------------------------------
# Several new tokens.

EXTEND = [
    # prefix, new, hq, hkv, d, page, block, first, last, sink, causal
    ([2000], [5], 64, 8, 64, 16, 16, 0, 0, True, True),
    ([0, 100, 31, 700], [1, 4, 0, 3], 16, 8, 64, 7, 7, 0, 0, False, True),
    ([500, 40], [8, 7], 32, 8, 128, 64, 32, 10, 50, True, True),
    ([500, 40], [16, 9], 8, 2, 64, 16, 8, 0, 6, True, True),      # windows shorter than the draft
    ([300, 20], [30, 2], 2, 2, 64, 16, 4, 0, 0, False, False),    # not causal
    ([600, 0, 33], [64, 64, 1], 1, 1, 128, 8, 8, 0, 0, True, True),
    ([130], [100], 12, 12, 64, 32, 16, 0, 0, True, True),
    ([1000, 3, 0, 200], [40, 33, 48, 0], 64, 8, 64, 16, 16, 0, 0, True, True),  # expanded from here on: chains
    ([700, 90], [37, 48], 16, 1, 64, 24, 8, 20, 61, False, True),
    ([500, 0, 33], [90, 96, 1], 32, 8, 128, 64, 32, 0, 0, True, True),
    ([900, 300], [80, 33], 24, 4, 128, 7, 7, 100, 30, True, True),
    ([1000, 3, 0, 200], [300, 129, 128, 0], 8, 2, 64, 16, 16, 0, 0, True, True),
    ([1000, 0], [200, 500], 8, 4, 128, 24, 8, 0, 0, False, True),
    ([2000, 700], [150, 400], 16, 4, 64, 16, 16, 100, 300, True, True),
    ([3000], [260], 4, 2, 128, 7, 7, 130, 513, False, True),
    ([200, 0], [130, 70], 8, 8, 64, 64, 64, 0, 0, True, False),
]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("case", EXTEND, ids=lambda c: f"n{max(c[1])}hq{c[2]}-{c[3]}d{c[4]}p{c[5]}w{c[7]}-{c[8]}")
def test_extend_matches_definition(ext, case, fmt):
    prefix, new, hq, hkv, d, page, block, first, last, sink, causal = case
    total = [p + n for p, n in zip(prefix, new)]
    c = Cache(total, hkv, d, page, block, fmt, seed=sum(new))
    g = torch.Generator().manual_seed(3)
    q = torch.randn(sum(new), hq, d, generator=g).bfloat16()
    sk = torch.rand(hq, generator=g) * 6 - 2 if sink else None
    out, lse = ext.attn_sink_fwd_paged_q8(q.cuda(), *c.dev(), cu(new).cuda(), torch.tensor(total).int().cuda(), max(new),
                                          max(total), None if sk is None else sk.cuda(), first, last, causal=causal)
    assert ext.device_status() == 0
    w = 2.0 ** -11 if max(new) * (hq // hkv) <= 64 else 2.0 ** -8
    at = 0
    for b, n in enumerate(new):
        k, v = c.tokens(b)
        check(out[at:at + n].cpu(), lse[:, at:at + n].cpu(), q[at:at + n], k, v, so.chunk_seen(total[b], n, first, last, causal),
              None if sk is None else sk.numpy(), w)
        at += n


@pytest.mark.parametrize("requests,hq,most,fmt", [(450, 7, 1, "e4m3"), (420, 7, 1, "int8"), (80, 14, 4, "e4m3"), (70, 30, 2, "int8")])
def test_many_rows_of_a_few_splits(ext, requests, hq, most, fmt):
    """Batches whose rows each have their splits merged by one warp: requests of several splits among short
    ones, ones without tokens and ones without rows, query heads that are no multiple of four."""
    rng = np.random.default_rng(requests)
    total = rng.integers(0, 200, requests)
    total[:8] = [9000, 0, 6001, 2049, 1, 257, 4096, 8999]
    new = np.minimum(rng.integers(0, most + 1, requests), total) if most > 1 else np.ones(requests, int)
    new[:8] = [most, 0 if most > 1 else 1, most, most, 1, most, most, most]
    c = Cache(total.tolist(), 1, 64, 16, 8, fmt, seed=requests)
    g = torch.Generator().manual_seed(4)
    q = torch.randn(int(new.sum()), hq, 64, generator=g).bfloat16()
    sk = torch.rand(hq, generator=g) * 6 - 2
    lens = torch.from_numpy(total).int().cuda()
    for sink in (None, sk):
        s = None if sink is None else sink.cuda()
        if most == 1:
            out, lse = ext.attn_sink_decode_paged_q8(q.cuda(), *c.dev(), lens, s)
            lse = lse.t()
        else:
            out, lse = ext.attn_sink_fwd_paged_q8(q.cuda(), *c.dev(), cu(new.tolist()).cuda(), lens, most, int(total.max()), s)
        assert ext.device_status() == 0
        full = [so.expand(x.numpy(), z.numpy(), fmt) for x, z in zip(c.codes, c.scales)]
        for b in list(range(8)) + rng.integers(8, requests, 20).tolist():
            at, n, t = int(new[:b].sum()), int(new[b]), np.arange(total[b])
            k, v = (x[c.table[b].numpy()[t // 16], t % 16] for x in full)
            if n:
                check(out[at:at + n].cpu(), lse[:, at:at + n].cpu(), q[at:at + n], k, v, so.chunk_seen(int(total[b]), n, 0, 0),
                      None if sink is None else sink.numpy(), 2.0 ** -11)


@pytest.mark.parametrize("n,hq", [(5, 4), (40, 32), (200, 4)])
def test_extend_leaves_other_rows_alone(ext, n, hq):
    """Rows behind the last request's and rows past max_seqlen_q stay; requests with fewer tokens
    than rows see none in the first ones.  (5 and 4: the row kernel, 40 and 32: chains, 200: the forward.)"""
    c = Cache([300, 3], 2, 64, 16, 16, "int8", seed=12)
    q = torch.randn(n + 5 + 4, hq, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    out = torch.full_like(q, 7).cuda()
    lse = torch.full((hq, q.shape[0]), 7.0).cuda()
    ext.device_status()
    ext.attn_sink_fwd_paged_q8(q.cuda(), *c.dev(), cu([n, 5]).cuda(), torch.tensor([300, 3]).int().cuda(), n, 300, out=out, lse=lse)
    assert ext.device_status() == 0
    assert torch.all(out[n + 5:] == 7) and torch.all(lse[:, n + 5:] == 7)
    for b, (lo, m) in enumerate(((0, n), (n, 5))):
        k, v = c.tokens(b)
        seen = so.chunk_seen(c.lens[b], m)
        check(out[lo:lo + m].cpu(), lse[:, lo:lo + m].cpu(), q[lo:lo + m], k, v, seen, None, 2.0 ** -8)
    assert torch.all(out[n:n + 2] == 0) and torch.all(lse[:, n:n + 2] == float("-inf"))


@pytest.mark.parametrize("n", [5, 40, 60])
def test_extend_of_more_tokens_than_the_table_holds(ext, n):
    """Lengths are cut at the table's 48 tokens (which end inside a tile) and reported, in all forms:
    the row kernel, a chain and the forward."""
    c = Cache([48, 48], 1, 64, 16, 16, "e4m3", seed=31)
    c.table = c.table[:, :3].contiguous()
    hq = 8
    q = torch.randn(2 * n, hq, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    junk = torch.full((64 << 20,), float("nan"), device="cuda")  # (memory that a later allocation may find)
    del junk
    ext.device_status()
    out, lse = ext.attn_sink_fwd_paged_q8(q.cuda(), *c.dev(), cu([n, n]).cuda(), torch.tensor([60, 48]).int().cuda(), n, 64)
    assert ext.device_status() == ext._lib.DEV_SEQLEN_OOB
    for b in range(2):
        k, v = c.tokens(b)
        rows = slice(b * n, (b + 1) * n)
        check(out[rows].cpu(), lse[:, rows].cpu(), q[rows], k, v, so.chunk_seen(48, n), None, 2.0 ** -8)


def test_expanded_batches_go_in_rounds(ext):
    """A length bound far above the lengths: scratch stays at 2 GiB and a little, results the same.
    (140 rows a request: the expanding form whatever the bound; fewer may go either way by it.)"""
    lens = [200 + 31 * b for b in range(24)]
    c = Cache(lens, 8, 128, 16, 16, "e4m3", seed=13)
    wide = torch.full((24, 65536 // 16), -1, dtype=torch.int32)
    wide[:, :c.table.shape[1]] = c.table
    q = torch.randn(24 * 140, 8, 128, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    dev, sl, cq = c.dev(), torch.tensor(lens).int().cuda(), cu([140] * 24).cuda()
    out, lse = ext.attn_sink_fwd_paged_q8(q, *dev, cq, sl, 140, max(lens))
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    dev[4] = wide.cuda()
    out2, lse2 = ext.attn_sink_fwd_paged_q8(q, *dev, cq, sl, 140, 65536)
    torch.cuda.synchronize()
    assert free - torch.cuda.mem_get_info()[0] <= 2400 << 20
    assert same(out, out2) and same(lse, lse2) and ext.device_status() == 0


def test_offsets_past_32_bits(ext):
    """A cache of more than 2^32 code bytes whose requests sit at its end."""
    page, hkv, d = 128, 64, 128
    pool = (1 << 32) // (page * hkv * d) + 4
    k = torch.zeros(pool, page, hkv, d, dtype=torch.int8, device="cuda")
    v = torch.zeros_like(k)
    ks, vs = (torch.ones(pool, 1, hkv, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(1)
    table = torch.tensor([[pool - 1, pool - 3]]).int()
    x = [torch.randn(200, hkv, d, generator=g).bfloat16() for _ in range(2)]
    sl = torch.tensor([200]).int().cuda()
    ext.attn_sink_kv_append_q8(*[t.cuda() for t in x], k, v, ks, vs, table.cuda(), sl, cu_new=cu([200]).cuda(), max_new=200)
    q = torch.randn(2, hkv, d, generator=g).bfloat16()
    out, lse = ext.attn_sink_fwd_paged_q8(q.cuda(), k, v, ks, vs, table.cuda(), cu([2]).cuda(), sl, 2, 200)
    cq = torch.randn(100, hkv, d, generator=g).bfloat16()
    cout, clse = ext.attn_sink_fwd_paged_q8(cq.cuda(), k, v, ks, vs, table.cuda(), cu([100]).cuda(), sl, 100, 200)
    assert ext.device_status() == 0 and int(k[:pool - 3].any()) == 0
    kk, vv = (so.expand(c[[pool - 1, pool - 3]].cpu().view(torch.uint8).numpy(), s[[pool - 1, pool - 3]].cpu().numpy(), "int8")
              .reshape(-1, hkv, d)[:200] for c, s in ((k, ks), (v, vs)))
    hs = slice(60, 64)
    check(out[:, hs].cpu(), lse[hs].cpu(), q[:, hs], kk[:, hs], vv[:, hs], so.chunk_seen(200, 2), None, 2.0 ** -11)
    check(cout[:, hs].cpu(), clse[hs].cpu(), cq[:, hs], kk[:, hs], vv[:, hs], so.chunk_seen(200, 100), None, 2.0 ** -8)


def test_calls_repeat_bit_for_bit(ext):
    c = Cache([5000, 333], 8, 64, 16, 16, "e4m3", seed=20)
    q = torch.randn(2, 64, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    dev, sl = c.dev(), torch.tensor([5000, 333]).int().cuda()
    a = ext.attn_sink_decode_paged_q8(q, *dev, sl)
    b = ext.attn_sink_decode_paged_q8(q, *dev, sl)
    assert same(a[0], b[0]) and same(a[1], b[1])
