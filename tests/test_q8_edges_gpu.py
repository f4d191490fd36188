"""The 8-bit attention where callers go to its ends: queries that are not numbers, scales far apart, more rows
than announced, windows over requests with fewer tokens than rows, chains in rounds.

Tolerances are those of test_q8_gpu.py; where V's scales lie 2^100 apart a weight's exponent is a number up to
2^7, whose roundings (half a step of 2^-17 of the exponent, of its difference from the reference, and lg2's
2^-22) change it by at most ln 2 (2^-18 + 2^-18 + 2^-22) < 2^-17, relative."""
import numpy as np
import pytest
import torch

from oracle import cache_ops_oracle as co
from oracle import serving_oracle as so
from cache_ops import cu, same
from test_q8_gpu import Cache, check, ext  # noqa: F401  (ext: the fixture)

pytestmark = pytest.mark.gpu
NAN = float("nan")


def lens_of(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("sink", [False, True])
@pytest.mark.parametrize("lens,new", [([100, 40], 1), ([1500, 900], 1), ([30000] + [64] * 70, 1), ([100, 40], 3), ([20000] + [64] * 70, 4)])
def test_queries_that_are_not_numbers_show(ext, lens, new, sink, fmt):  # noqa: F811
    """A NaN in a row's query makes its output and lse NaN (not the empty row's 0 and -inf), and no other's:
    one CTA a row, splits merged as a cluster, and by a launch of their own."""
    c = Cache(lens, 2, 64, 16, 16, fmt, seed=4)
    g = torch.Generator().manual_seed(3)
    q = torch.randn(len(lens) * new, 8, 64, generator=g).bfloat16()
    bad = q.clone()
    where = torch.zeros(q.shape[:2], dtype=torch.bool)
    for row, head, dim in ((0, 0, slice(None)), (0, 6, 17), (new, 3, 63)):
        bad[row, head, dim] = NAN
        where[row, head] = True
    sk = torch.rand(8, generator=g).cuda() if sink else None
    dev, sl, c_q = c.dev(), lens_of(lens), cu([new] * len(lens)).cuda()

    def call(x):
        if new == 1:
            return ext.attn_sink_decode_paged_q8(x.cuda(), *dev, sl, sk)
        out, lse = ext.attn_sink_fwd_paged_q8(x.cuda(), *dev, c_q, sl, new, max(lens), sk)
        return out, lse.t().contiguous()

    (out, lse), (good, good_lse) = call(bad), call(q)
    where = where.cuda()
    assert torch.all(torch.isnan(out[where])) and torch.all(torch.isnan(lse[where]))
    # (the references that others move to may differ, and with them the last bits: twice the tolerance, A <= max |v|)
    out, good_out, most = out[~where].float(), good[~where].float(), float(c.scales[1].max()) * so.QMAX[fmt]
    assert torch.all((out - good_out).abs() <= 2.0 ** -7 * good_out.abs() + 2.0 ** -9 * most)
    assert torch.all((lse[~where] - good_lse[~where]).abs() <= 2.0 ** -9)
    assert not torch.any(torch.isnan(good)) and ext.device_status() == 0


@pytest.mark.parametrize("apart", [24, 28, 30])
def test_weights_beside_much_larger_scales(ext, apart):  # noqa: F811
    """Blocks of V's scale 2^apart whose codes are 0 in the upper dims, where only the other blocks (scale 1)
    count: their weights are off by 2^-11 of each or 2^-32 of the largest, times the V scales, whichever is more."""
    n, d, block = 512, 64, 16
    c = Cache([n], 1, d, 16, block, "int8", seed=apart, spread=0)
    t = np.arange(n)
    page = c.table[0].numpy()[t // 16]
    large = (t // block) % 2 == 0
    c.scales[0][:] = 2.0 ** -9
    c.scales[1][:] = 1.0
    c.scales[1][page[large]] = 2.0 ** apart
    codes = c.codes[1].view(torch.int8)
    for p in np.unique(page[large]):
        codes[p, :, :, 32:] = 0
    q = torch.randn(1, 4, d, generator=torch.Generator().manual_seed(1)).bfloat16()
    out, lse = ext.attn_sink_decode_paged_q8(q.cuda(), *c.dev(), lens_of([n]))
    k, v = c.tokens(0)
    O, L, P, A = co.attend(q, k, v, np.ones((1, n), bool), None, d ** -0.5)
    P = np.asarray(P).reshape(4, n)
    vs = np.where(large, 2.0 ** apart, 1.0)
    off = np.maximum(2.0 ** -11 * P * vs, 2.0 ** -32 * (P * vs).max(1, keepdims=True))
    bound = np.einsum("ht,td->hd", off / vs, np.abs(v[:, 0]))
    S = d ** -0.5 * np.abs(co.to_np(q)).max() * np.abs(k).sum(-1).max()
    delta = (d + 8) * 2.0 ** -24 * S
    err = np.abs(co.to_np(out)[0] - O[0])
    assert np.all(err <= 2.0 ** -8 * np.abs(O[0]) + bound + (2 * delta + 2.0 ** -17) * A[0])
    assert np.all(np.abs(co.to_np(lse)[0] - L[:, 0]) <= delta + 2.0 ** -17)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("new", [1, 4])
def test_scales_of_v_up_to_two_to_the_hundred_apart(ext, new, fmt):  # noqa: F811
    """The denominator and lse know nothing of V's scales."""
    n, d = 700, 64
    c = Cache([n], 2, d, 16, 16, fmt, seed=9)
    g = torch.Generator().manual_seed(9)
    c.scales[1] = torch.exp2(50.0 * (torch.randint(0, 2, c.scales[1].shape, generator=g) * 2 - 1))
    q = torch.randn(new, 8, d, generator=g).bfloat16()
    out, lse = ext.attn_sink_fwd_paged_q8(q.cuda(), *c.dev(), cu([new]).cuda(), lens_of([n]), new, n)
    k, v = c.tokens(0)
    O, L, P, A = co.attend(q, k, v, so.chunk_seen(n, new), None, d ** -0.5)
    S = d ** -0.5 * np.abs(co.to_np(q)).max() * np.abs(k).sum(-1).max()
    delta = (d + 8) * 2.0 ** -24 * S
    assert np.all(np.abs(co.to_np(lse) - L) <= delta + 2.0 ** -17)
    assert np.all(np.abs(co.to_np(out) - O) <= 2.0 ** -8 * np.abs(O) + (2.0 ** -11 + 2 * delta + 2.0 ** -16) * A)


@pytest.mark.parametrize("n,most,hq", [(9, 5, 4), (60, 40, 32), (400, 200, 4)])
def test_more_rows_than_announced(ext, n, most, hq):  # noqa: F811
    """A request of n rows where max_seqlen_q is fewer, in the row kernel, as a chain and in the forward: reported; the
    rows up to the bound are right at their uncut positions, as are the other request's, and the rows behind both
    requests stay.  (Those past the bound stay where the path goes by rows.)"""
    lens, rows = [500, 300], [n, most - 1]
    c = Cache(lens, 2, 64, 16, 16, "e4m3", seed=12)
    q = torch.randn(sum(rows) + 3, hq, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    for first, last in ((0, 0), (20, 70)):
        out, lse = torch.full_like(q, 7).cuda(), torch.full((hq, q.shape[0]), 7.0).cuda()
        ext.device_status()
        ext.attn_sink_fwd_paged_q8(q.cuda(), *c.dev(), cu(rows).cuda(), lens_of(lens), most, 500, None, first, last, out=out, lse=lse)
        assert ext.device_status() == ext._lib.DEV_SEQLEN_OOB
        assert torch.all(out[sum(rows):] == 7) and torch.all(lse[:, sum(rows):] == 7)
        if most < 128:
            assert torch.all(out[most:n] == 7) and torch.all(lse[:, most:n] == 7)
        k, v = c.tokens(0)
        seen = so.chunk_seen(500, n, first, last)[:most]
        check(out[:most].cpu(), lse[:, :most].cpu(), q[:most], k, v, seen, None, 2.0 ** -8)
        k, v = c.tokens(1)
        at = slice(n, sum(rows))
        check(out[at].cpu(), lse[:, at].cpu(), q[at], k, v, so.chunk_seen(300, most - 1, first, last), None, 2.0 ** -8)


@pytest.mark.parametrize("n,hq,d", [(6, 4, 64), (40, 32, 64), (90, 32, 128), (200, 4, 64)])
@pytest.mark.parametrize("first,last", [(0, 3), (4, 9), (2, 500)])
def test_windows_over_fewer_tokens_than_rows(ext, n, hq, d, first, last):  # noqa: F811
    """Requests whose first rows stand before position 0 and see nothing, under a window, in each path."""
    lens = [n - 3, 1, 0, n // 2]
    c = Cache(lens, 2, d, 16, 16, "int8", seed=n)
    q = torch.randn(4 * n, hq, d, generator=torch.Generator().manual_seed(2)).bfloat16()
    out, lse = ext.attn_sink_fwd_paged_q8(q.cuda(), *c.dev(), cu([n] * 4).cuda(), lens_of(lens), n, max(lens), None, first, last)
    assert ext.device_status() == 0
    for b, length in enumerate(lens):
        at = slice(b * n, (b + 1) * n)
        k, v = c.tokens(b)
        check(out[at].cpu(), lse[:, at].cpu(), q[at], k, v, so.chunk_seen(length, n, first, last), None, 2.0 ** -8)
        none = max(0, n - length)
        assert torch.all(out[at][:none] == 0) and torch.all(lse[:, at][:, :none] == float("-inf"))


@pytest.mark.parametrize("first,last", [(0, 0), (30, 100)])
def test_chains_go_in_rounds(ext, first, last):  # noqa: F811
    """Chains whose expanded tokens do not fit the scratch together: requests of every round, ones with no rows
    among them, against the definition."""
    lens = [150 + 37 * b for b in range(24)]
    rows = [(b * 7) % 41 for b in range(24)]
    c = Cache(lens, 8, 64, 16, 16, "e4m3", seed=13)
    wide = torch.full((24, 65536 // 16), -1, dtype=torch.int32)
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    q = torch.randn(sum(rows), 64, 64, generator=torch.Generator().manual_seed(1)).bfloat16()
    sk = torch.rand(64, generator=torch.Generator().manual_seed(2)) * 4
    # 24 requests of up to 65536 tokens at 2 KB each: 3.2 GB
    out, lse = ext.attn_sink_fwd_paged_q8(q.cuda(), *c.dev(), cu(rows).cuda(), lens_of(lens), 40, 65536, sk.cuda(), first, last)
    assert ext.device_status() == 0
    at = 0
    for b, n in enumerate(rows):
        if n and b in (1, 2, 5, 11, 12, 13, 20, 23):
            k, v = c.tokens(b)
            check(out[at:at + n].cpu(), lse[:, at:at + n].cpu(), q[at:at + n], k, v, so.chunk_seen(lens[b], n, first, last), sk.numpy(), 2.0 ** -8)
        at += n


def test_bounds_above_int32_are_no_bounds(ext):  # noqa: F811
    """A length bound that no int holds is taken as none; more rows than one call takes are refused."""
    c = Cache([90, 40], 2, 64, 16, 16, "e4m3", seed=1)
    q = torch.randn(10, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    args = (q, *c.dev(), cu([6, 4]).cuda(), lens_of([90, 40]))
    want = ext.attn_sink_fwd_paged_q8(*args, 6, 2 ** 31 - 1)
    for bound in (2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 40):
        got = ext.attn_sink_fwd_paged_q8(*args, 6, bound)
        assert same(got[0], want[0]) and same(got[1], want[1])
        with pytest.raises(RuntimeError):
            ext.attn_sink_fwd_paged_q8(*args, bound, 90)
    assert ext.device_status() == 0
