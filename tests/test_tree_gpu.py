"""Attention of drafted trees over a paged cache against the fp64 definition.

Tolerances: the weights P are rounded to bf16 before P V (2^-8 of each) and the
output once more (2^-8 of its value), so |O - O*| <= 2^-8 (sum P |v| + |O*|); the
fp32 scores, exponentials and sums add less than 2^-13 of sum P |v|.  LSE is off by
no more than the largest score: d + 8 fp32 roundings (2^-24) of sum |q k| scale
(below 15 for these inputs), 1.3e-4, and the exponentials' 2^-21."""
import numpy as np
import pytest
import torch

from oracle import cache_ops_oracle as co
from cache_ops import cu, paged, same

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ext():
    from paged_kv_sink_gb300 import build
    build.build()
    import paged_kv_sink_gb300 as ext
    return ext


def make(prefix, nodes, hq, hkv, d, page, seed=0, sink=True, kind="random"):
    k_cache, v_cache, table, sl = paged([p + n for p, n in zip(prefix, nodes)], hkv, d, page, seed)
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn(sum(nodes), hq, d, generator=g).bfloat16()
    sk = torch.rand(hq, generator=g) * 6 - 2 if sink else None
    parents = []
    for n in nodes:
        if kind == "chain":
            parents += list(range(-1, n - 1))
        elif kind == "roots":
            parents += [-1] * n
        else:
            parents += [int(torch.randint(-1, i, (1,), generator=g)) if i else -1 for i in range(n)]
    return dict(q=q, k=k_cache, v=v_cache, table=table, sl=sl, cu=cu(nodes), parents=torch.tensor(parents).int(),
                sink=sk, prefix=prefix, nodes=nodes)


def run(ext, x, first=0, last=0, scale=0.0, max_k=None, **kw):
    dev = {n: None if x[n] is None else x[n].cuda() for n in ("q", "k", "v", "table", "sl", "cu", "parents", "sink")}
    out, lse = ext.attn_sink_tree_paged(dev["q"], dev["k"], dev["v"], dev["table"], dev["cu"], dev["sl"],
                                        dev["parents"], max(x["nodes"] + [0]), max_k or int(max(x["sl"])),
                                        sink=dev["sink"], win_first=first, win_last=last, scale=scale, **kw)
    torch.cuda.synchronize()
    return out.cpu(), None if lse is None else lse.cpu()


def check(x, out, lse, first=0, last=0, scale=0.0, requests=None):
    row, d = 0, x["q"].shape[2]
    for b, (p, n) in enumerate(zip(x["prefix"], x["nodes"])):
        if n and (requests is None or b in requests):
            seen = co.tree_seen(x["parents"][row:row + n].tolist(), p, first, last)
            used = np.nonzero(seen.any(0))[0]
            k, v = (co.tokens(x[c], x["table"][b], p + n)[used] for c in ("k", "v"))
            O, L, _, A = co.attend(x["q"][row:row + n], k, v, seen[:, used],
                                   None if x["sink"] is None else x["sink"].numpy(), scale or d ** -0.5)
            err = np.abs(co.to_np(out[row:row + n]) - O)
            bound = 2.0 ** -8 * (A + np.abs(O)) + 2.0 ** -13 * A
            assert np.all(err <= bound), (b, float((err - bound).max()))
            np.testing.assert_allclose(lse[:, row:row + n].numpy(), L, atol=1.5e-4)
        row += n


CASES = [
    # prefix, nodes, hq, hkv, d, page, first, last, kind
    ([40], [1], 8, 1, 64, 16, 0, 0, "random"),
    ([0, 1, 127, 128, 129], [5, 1, 1, 2, 3], 8, 2, 64, 16, 0, 0, "random"),     # empty and tile-edge prefixes
    ([500, 3, 1000], [17, 64, 33], 16, 2, 64, 8, 0, 0, "random"),
    ([300, 0], [256, 200], 8, 2, 64, 128, 0, 0, "random"),                      # the largest trees
    ([200], [130], 4, 4, 64, 32, 0, 0, "chain"),                                # group 1, nodes past one tile
    ([90, 700], [16, 5], 12, 2, 128, 64, 0, 0, "roots"),                        # group 6
    ([250], [40], 20, 1, 64, 16, 0, 0, "random"),                               # group 20
    ([64, 300], [9, 30], 40, 1, 128, 16, 0, 0, "random"),                       # group 40
    ([30], [7], 128, 1, 64, 16, 0, 0, "random"),                                # group 128: one node a tile
    ([2000, 10], [24, 12], 16, 2, 64, 16, 100, 300, "random"),                  # windows with a gap
    ([600, 129], [20, 40], 8, 2, 128, 64, 4, 9, "chain"),                       # ancestors leave the window
    ([600], [20], 8, 2, 64, 16, 0, 1, "chain"),                                 # each sees itself alone
    ([900], [6], 8, 2, 64, 256, 0, 128, "random"),                              # pages above a tile
    ([9000], [12], 64, 8, 64, 16, 1024, 7168, "random"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"p{max(c[0])}n{max(c[1])}hq{c[2]}-{c[3]}d{c[4]}w{c[6]}-{c[7]}{c[8]}")
def test_tree_matches_definition(ext, case):
    prefix, nodes, hq, hkv, d, page, first, last, kind = case
    x = make(prefix, nodes, hq, hkv, d, page, seed=len(nodes) + hq, kind=kind)
    out, lse = run(ext, x, first, last)
    assert ext.device_status() == 0
    check(x, out, lse, first, last)


def test_without_sink_with_scale_and_wrong_length_estimates(ext):
    x = make([300, 2500, 77], [4, 19, 8], 8, 2, 64, 16, sink=False)
    out, lse = run(ext, x, scale=0.3)
    check(x, out, lse, scale=0.3)
    for max_k in (1, 100000):  # plans the split only
        out, lse = run(ext, x, scale=0.3, max_k=max_k)
        check(x, out, lse, scale=0.3)
    out, none = run(ext, x, scale=0.3, return_lse=False)
    assert none is None


def test_many_requests_and_no_nodes(ext):
    g = torch.Generator().manual_seed(5)
    prefix = torch.randint(0, 400, (40,), generator=g).tolist()
    nodes = torch.randint(0, 12, (40,), generator=g).tolist()
    x = make(prefix, nodes, 8, 2, 64, 16, seed=6)
    out, lse = run(ext, x)
    check(x, out, lse)
    x = make([10], [0], 8, 2, 64, 16)
    assert run(ext, x)[0].shape == (0, 8, 64)


@pytest.mark.parametrize("hq,hkv,d", [(160, 160, 128), (320, 320, 64), (301, 301, 64)])
def test_more_kv_heads_than_resident_blocks(ext, hq, hkv, d):
    x = make([140, 20], [3, 2], hq, hkv, d, 16, seed=17)
    out, lse = run(ext, x)
    check(x, out, lse)


def test_more_requests_than_threads(ext):
    """The shares of the batch are found 256 requests at a time."""
    g = torch.Generator().manual_seed(6)
    prefix = torch.randint(0, 200, (600,), generator=g).tolist()
    nodes = [n if b % 7 else 0 for b, n in enumerate(torch.randint(0, 4, (600,), generator=g).tolist())]
    x = make(prefix, nodes, 4, 1, 64, 16, seed=18)
    out, lse = run(ext, x)
    check(x, out, lse)


def test_a_chain_equals_the_paged_forward(ext):
    x = make([700, 33], [60, 130], 16, 2, 64, 16, kind="chain")
    for first, last in ((0, 0), (20, 100)):
        out, lse = run(ext, x, first, last)
        ref, ref_lse = ext.attn_sink_fwd_paged(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), x["table"].cuda(),
                                               x["cu"].cuda(), x["sl"].cuda(), 130, int(max(x["sl"])),
                                               sink=x["sink"].cuda(), win_first=first, win_last=last)
        check(x, out, lse, first, last)
        check(x, ref.cpu(), ref_lse.cpu(), first, last)


@pytest.mark.parametrize("sink", [80.0, float("inf"), float("-inf"), -50.0])
def test_sink_limits(ext, sink):
    x = make([50, 400], [3, 9], 8, 2, 64, 16)
    x["sink"] = torch.full((8,), sink)
    out, lse = run(ext, x)
    if sink == float("inf"):
        assert torch.all(out == 0) and torch.all(torch.isposinf(lse))
    else:
        if sink == float("-inf"):
            x["sink"] = None
        check(x, out, lse)


def test_large_scores(ext):
    """Scores of a few hundred that grow along the keys: the running maximum moves often.
    The fp32 score error grows with sum |q k| scale (60 times the usual): LSE 1e-2, and the
    weights by the same factor e^(2 * 1e-2)."""
    x = make([600], [10], 8, 2, 64, 16, seed=9)
    rows = x["k"].view(-1, 2, 64)
    for t in range(610):
        rows[int(co.slot(x["table"][0].numpy(), 16, [t])[0])] *= 0.05 * (t % 300)
    x["q"] *= 4
    out, lse = run(ext, x)
    seen = co.tree_seen(x["parents"].tolist(), 600)
    k, v = (co.tokens(x[c], x["table"][0], 610) for c in ("k", "v"))
    O, L, _, A = co.attend(x["q"], k, v, seen, x["sink"].numpy(), 0.125)
    np.testing.assert_allclose(lse.numpy(), L, atol=1e-2)
    assert np.all(np.abs(co.to_np(out) - O) <= 2.0 ** -8 * (A + np.abs(O)) + 2.1e-2 * A)


def test_many_requests_of_one_node(ext):
    """More requests than one block scans, of lengths that the runs cut anywhere."""
    x = make([(37 * i) % 900 for i in range(300)], [1] * 300, 8, 1, 64, 16, seed=3)
    out, lse = run(ext, x)
    assert ext.device_status() == 0
    check(x, out, lse)


@pytest.mark.parametrize("prefix,nodes,hq,d,page,first,last", [
    ([1000 + 7 * i for i in range(30)], [20 + i % 13 for i in range(30)], 64, 64, 16, 0, 0),   # short row tiles
    ([9000, 3000], [100, 60], 64, 64, 16, 0, 0),                                               # over many runs
    ([2000 + 50 * i for i in range(12)], [40] * 12, 32, 128, 64, 64, 900),
    ([300 + 90 * i for i in range(24)], [70] * 24, 32, 128, 16, 0, 0)])
def test_row_tiles_that_runs_cut(ext, prefix, nodes, hq, d, page, first, last):
    """Several row tiles a request, cut by the GPU's runs at many places: each takes every key tile once."""
    x = make(prefix, nodes, hq, 8, d, page, seed=14)
    out, lse = run(ext, x, first, last)
    assert ext.device_status() == 0
    check(x, out, lse, first, last)


@pytest.mark.parametrize("prefix", [50, 2000])
def test_infinite_scores_give_nan(ext, prefix):
    """A visible token with a score of +inf leaves no finite softmax, however the keys are split."""
    x = make([prefix], [5], 8, 2, 64, 16, seed=6)
    x["q"] = x["q"].abs() + 0.5
    x["k"].view(-1, 2, 64)[co.slot(x["table"][0].numpy(), 16, 20)] = float("inf")
    out, lse = run(ext, x)
    assert torch.all(torch.isnan(out)) and not torch.any(torch.isfinite(lse))


def test_rows_of_other_requests_stay(ext):
    """Rows of out and lse behind the last request's keep what they held."""
    x = make([30], [5], 8, 2, 64, 16)
    q = torch.cat([x["q"], torch.full((4, 8, 64), float("nan")).bfloat16()])
    out, lse = torch.full((9, 8, 64), 3.0).bfloat16().cuda(), torch.full((8, 9), 3.0).cuda()
    y = dict(x, q=q, parents=torch.cat([x["parents"], torch.full((4,), -7).int()]))
    run(ext, y, out=out, lse=lse)
    assert ext.device_status() == 0
    check(x, out.cpu()[:5], lse.cpu()[:, :5])
    assert torch.all(out[5:] == 3) and torch.all(lse[:, 5:] == 3)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
def test_infinities_and_nans_reach_only_who_sees_them(ext, d, page):
    """A drafted token whose K or V holds infinities or NaNs changes its descendants
    alone; tokens in the window's gap change nobody."""
    nodes = 40
    x = make([300], [nodes], 8, 2, d, page, seed=13, sink=True)
    first, last = 10, 120                       # the gap: tokens 10 .. 180
    want, want_lse = run(ext, x, first, last)
    seen = co.tree_seen(x["parents"].tolist(), 300, first, last)
    for t in range(10, 180):
        s = co.slot(x["table"][0].numpy(), page, t)
        x["k"].view(-1, 2, d)[s] = float("nan")
        x["v"].view(-1, 2, d)[s] = float("inf")
    out, lse = run(ext, x, first, last)
    assert same(out, want) and same(lse, want_lse)
    v = x["v"].view(-1, 2, d)
    at = [int(co.slot(x["table"][0].numpy(), page, 300 + i)) for i in range(nodes)]
    v[at[5], 0, 3], v[at[7], 1, 60], v[at[9], 0, 3] = float("inf"), float("nan"), float("-inf")
    # a prefix token that the window shows to nodes of depth 0 and 1 only
    v[int(co.slot(x["table"][0].numpy(), page, 182)), 0, 40] = float("inf")
    assert 0 < seen[:, 182].sum() < nodes
    out, lse = run(ext, x, first, last)
    assert same(lse, want_lse)
    for i in range(nodes):
        for h in range(8):
            row = want[i, h].clone()
            if h < 4 and seen[i, 305]:
                row[3] = float("inf")
            if h < 4 and seen[i, 309]:
                row[3] = float("nan") if seen[i, 305] else float("-inf")
            if h < 4 and seen[i, 182]:
                row[40] = float("inf")
            if h >= 4 and seen[i, 307]:
                row[60] = float("nan")
            assert torch.equal(row.isnan(), out[i, h].isnan()), (i, h)
            assert torch.equal(row.nan_to_num(7.0, 8.0, 9.0), out[i, h].nan_to_num(7.0, 8.0, 9.0)), (i, h)
    x["k"].view(-1, 2, d)[at[11], 1] = float("nan")
    out2, lse2 = run(ext, x, first, last)
    for i in range(nodes):
        keep = slice(0, 4) if seen[i, 311] else slice(0, 8)
        assert same(lse2[keep, i], lse[keep, i])
        if seen[i, 311]:
            assert torch.all(lse2[4:, i].isnan())


def test_bad_parents_pages_and_lengths_raise_status(ext):
    x = make([60, 60, 60], [6, 6, 6], 8, 2, 64, 16)
    ext.device_status()
    y = dict(x, parents=x["parents"].clone())
    y["parents"][6:9] = torch.tensor([0, 1, -9])   # request 1: its own index, itself, below -1
    out, lse = run(ext, y)
    assert ext.device_status() == ext._lib.DEV_TREE
    y["parents"][6:9] = -1                         # is what they are read as
    check(y, out, lse)
    y = dict(x, table=x["table"].clone())
    y["table"][1, 1] = 10 ** 6
    out, lse = run(ext, y)
    assert ext.device_status() == ext._lib.DEV_PAGE_OOB
    check(x, out, lse, requests=(0, 2))
    # request 1 without its tokens 16..31: a prefix of 44 tokens with page 1 left out
    z = dict(x, table=x["table"].clone(), sl=x["sl"].clone(), prefix=[60, 44, 60])
    z["table"][1, 1:4] = x["table"][1, 2:5]
    z["sl"][1] = 50
    check(z, out, lse, requests=(1,))
    y = dict(x, sl=torch.tensor([66, 4, 10 ** 6]).int())
    out, lse = run(ext, y, max_k=100)
    assert ext.device_status() & ext._lib.DEV_SEQLEN_OOB
    check(x, out, lse, requests=(0,))
    assert torch.all(out[6:12] == 0) and torch.allclose(lse[:, 6:12], x["sink"][:, None])
    out = torch.full((18, 8, 64), 3.0).bfloat16().cuda()
    ext.device_status()
    run(ext, dict(x, nodes=[2, 2, 2]), out=out)    # the grid may cover more rows than max_seqlen_q, or not
    assert ext.device_status() == ext._lib.DEV_SEQLEN_OOB
    assert torch.all(out[2:6] == 3)


def test_two_graphs_and_two_streams(ext):
    """Two captured calls replayed on two streams at once, and an eager one between, do
    not share scratch."""
    xs = [make([900, 50], [12, 3], 16, 2, 64, 16, seed=s) for s in (20, 21)]
    names = ("q", "k", "v", "table", "sl", "cu", "parents", "sink")
    devs = [{n: x[n].cuda() for n in names} for x in xs]

    def call(d, out, lse):
        ext.attn_sink_tree_paged(d["q"], d["k"], d["v"], d["table"], d["cu"], d["sl"], d["parents"], 12, 912,
                                 sink=d["sink"], out=out, lse=lse)

    outs = [(torch.empty_like(d["q"]), torch.empty(16, 15, device="cuda")) for d in devs]
    graphs = []
    for d, o in zip(devs, outs):
        call(d, *o)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(d, *o)
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for o in outs:
            o[0].zero_(), o[1].zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = (torch.empty_like(devs[0]["q"]), torch.empty(16, 15, device="cuda"))
        call(devs[0], *eager)
        torch.cuda.synchronize()
        for x, o in zip(xs, outs):
            check(x, o[0].cpu(), o[1].cpu())
        assert same(eager[0], outs[0][0]) and same(eager[1], outs[0][1])


@pytest.mark.parametrize("hq,hkv,d,page", [(8, 2, 64, 16), (8, 2, 128, 64), (24, 8, 64, 8)])
def test_rows_of_a_warp_with_walks_of_different_lengths(ext, hq, hkv, d, page):
    """Neighbouring nodes at depths from 0 to 60: each row walks its own number of steps to
    its root, before a segment's first tile (positions, under a window), in masked tiles,
    and again between the pieces of the output where V holds infinities."""
    nodes, prefix = [90, 33, 120, 7], [400, 10, 129, 0]
    x = make(prefix, nodes, hq, hkv, d, page, seed=23)
    parents = []
    for n in nodes:  # even nodes are a chain, every second odd one is a root, the others hang on the chain's start
        parents += [i - 2 if i % 2 == 0 and i else -1 if i % 4 != 3 else 0 for i in range(n)]
    x["parents"] = torch.tensor(parents).int()
    first, last = 6, 40
    out, lse = run(ext, x, first, last)
    assert ext.device_status() == 0
    check(x, out, lse, first, last)
    # an infinity in every 32 columns of the V rows of a chain's node and of a root
    v, row = x["v"].view(-1, hkv, d), 0
    for b, n in enumerate(nodes):
        for i in (4, 5):
            v[int(co.slot(x["table"][b].numpy(), page, prefix[b] + i)), :, i::32] = float("inf")
    got, got_lse = run(ext, x, first, last)
    assert ext.device_status() == 0 and same(got_lse, lse)
    for b, n in enumerate(nodes):
        seen = co.tree_seen(parents[row:row + n], prefix[b], first, last)
        want = out[row:row + n].clone()
        for i in (4, 5):
            sees = torch.from_numpy(np.nonzero(seen[:, prefix[b] + i])[0])
            want[sees[:, None], :, torch.arange(i, d, 32)[None]] = float("inf")
        assert same(got[row:row + n], want), b
        row += n


def test_length_estimates_change_nothing(ext):
    """max_seqlen_k is checked for its sign alone: the keys are split by the lengths on the
    device, so any estimate gives the same bits."""
    x = make([300, 2500, 77], [4, 19, 8], 8, 2, 64, 16)
    want, want_lse = run(ext, x, max_k=2519)
    check(x, want, want_lse)
    dev = {n: x[n].cuda() for n in ("q", "k", "v", "table", "sl", "cu", "parents", "sink")}
    args = [dev[n] for n in ("q", "k", "v", "table", "cu", "sl", "parents")]
    for max_k in (0, 1, 100000, 2 ** 31 - 1):
        out, lse = ext.attn_sink_tree_paged(*args, 19, max_k, sink=dev["sink"])
        assert same(out.cpu(), want) and same(lse.cpu(), want_lse)
    with pytest.raises(ext.AttnSinkError, match="sizes"):
        ext.attn_sink_tree_paged(*args, 19, -1, sink=dev["sink"])
