"""The 8-bit cache, verification and pages run together, as a server runs them: a speculative loop
over an 8-bit cache whose pages the library hands out, parallel samples over shared pages, a
step captured in a graph, and the same calls on other streams."""
import numpy as np
import pytest
import torch

from oracle import cache_ops_oracle as co
from oracle import serving_oracle as so
from cache_ops import cu, same

pytestmark = pytest.mark.gpu
HQ, HKV, D, PAGE, BLOCK, POOL, WIDTH = 8, 2, 64, 16, 8, 64, 16


@pytest.fixture(scope="module")
def ext():
    from paged_kv_sink_gb300 import build
    build.build()
    import paged_kv_sink_gb300 as ext
    return ext


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    def __init__(self, ext, rows, fmt, seed=0):
        self.ext, self.g = ext, torch.Generator(device="cuda").manual_seed(seed)
        kind = dict(e4m3=torch.float8_e4m3fn, int8=torch.int8)[fmt]
        self.cache = [torch.zeros(POOL, PAGE, HKV, D, dtype=torch.int8, device="cuda").view(kind) for _ in range(2)]
        self.cache += [torch.ones(POOL, PAGE // BLOCK, HKV, device="cuda") for _ in range(2)]
        self.table = torch.full((rows, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(POOL, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(rows, dtype=torch.int32, device="cuda")

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").bfloat16()

    def grow(self, new):
        missing = self.ext.attn_sink_pages_reserve(self.cache, self.table, self.refs, self.lens, new, PAGE)
        self.lens = new
        return missing

    def append(self, k, v, counts):
        self.ext.attn_sink_kv_append_q8(k, v, *self.cache, self.table, self.lens, cu_new=cu(counts).cuda(), max_new=max(counts))

    def extend(self, q, counts, **kw):
        return self.ext.attn_sink_fwd_paged_q8(q, *self.cache, self.table, cu(counts).cuda(), self.lens, max(counts), WIDTH * PAGE, **kw)

    def tokens(self, b):
        n = int(self.lens[b])
        t, row = np.arange(n), self.table[b].cpu().numpy()
        fmt = "int8" if self.cache[0].dtype == torch.int8 else "e4m3"
        return [so.expand(self.cache[i].cpu().view(torch.uint8).numpy(), self.cache[2 + i].cpu().numpy(), fmt)[row[t // PAGE], t % PAGE]
                for i in range(2)]

    def counts_agree(self):
        held = np.zeros(POOL, int)
        for row, n in zip(self.table.cpu().numpy(), self.lens.tolist()):
            np.add.at(held, row[:-(-n // PAGE)], 1)
        np.testing.assert_array_equal(held, self.refs.cpu().numpy())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_a_speculative_loop(ext, fmt):
    """Prompts, then drafts in a row: pages reserved, written, attended to, verified, and what was
    refused given back.  The cache keeps what a model of the accepted rows says, within a step of
    its codes; attention is what the cache's values give."""
    s, B, vocab, n = Server(ext, 3, fmt), 3, 700, 4
    counts = [30, 5, 17]
    s.grow(i32(counts))
    kept = [[s.normal(c, HKV, D) for c in counts] for _ in range(2)]
    s.append(torch.cat(kept[0]), torch.cat(kept[1]), counts)
    accepted = 0
    for step in range(6):
        prefix = s.lens
        assert int(s.grow(prefix + n)) == 0
        k, v, q = s.normal(B * n, HKV, D), s.normal(B * n, HKV, D), s.normal(B * n, HQ, D)
        s.append(k, v, [n] * B)
        out, lse = s.extend(q, [n] * B)
        logits = out.float().flatten(1) @ torch.randn(HQ * D, vocab, generator=s.g, device="cuda")
        p = (logits * 0.3).softmax(-1)
        dr = (logits * 0.3 + torch.randn(B * n, vocab, generator=s.g, device="cuda") * 0.3).softmax(-1)
        tok = torch.zeros(B, n, dtype=torch.int64, device="cuda")
        tok[:, 1:] = torch.multinomial(dr, 1, generator=s.g).view(B, n)[:, :-1]
        u, un = torch.rand(B * n, generator=s.g, device="cuda"), torch.rand(B, generator=s.g, device="cuda")
        src, cnt, following = ext.attn_sink_verify_draft(p, tok.int().flatten(), None, cu([n] * B).cuda(), u, un, n, draft=dr, base=prefix)
        for b in range(B):
            O, L, P, A = co.attend(q[b * n:(b + 1) * n], *s.tokens(b), so.chunk_seen(int(s.lens[b]), n), None, D ** -0.5)
            err = np.abs(co.to_np(out[b * n:(b + 1) * n]) - O)
            assert np.all(err <= 2.0 ** -8 * np.abs(O) + 2.0 ** -10 * A)
            path, token, _ = so.verify(co.to_np(p[b * n:(b + 1) * n]), co.to_np(dr[b * n:(b + 1) * n]), tok[b].tolist(), [-1, 0, 1, 2],
                                       u[b * n:(b + 1) * n].tolist(), float(un[b]))
            assert int(cnt[b]) == len(path) and int(following[b]) == token
            assert src[b].tolist() == [int(prefix[b]) + i for i in path] + [-1] * (n - len(path))
            for i, x in enumerate((k, v)):
                kept[i][b] = torch.cat([kept[i][b], x[b * n:b * n + len(path)]])
            accepted += len(path) - 1
        # in a row the tokens that stand are in place already: the rest is cut off
        ext.attn_sink_pages_release(s.table, s.refs, s.lens, prefix + cnt, PAGE)
        s.lens = prefix + cnt
        s.counts_agree()
    assert accepted > 0 and ext.device_status() == 0
    for b in range(B):
        for i, have in enumerate(s.tokens(b)):
            want = co.to_np(kept[i][b])
            t = np.arange(len(want))
            row = s.table[b].cpu().numpy()
            scale = s.cache[2 + i].cpu().double().numpy()[row[t // PAGE], t % PAGE // BLOCK][..., None]
            # (see test_serving_oracle.py: a block filled in several calls)
            bound = scale if fmt == "int8" else 2.0 ** -4 * np.abs(want) + 2.0 ** -9 * scale
            assert np.all(np.abs(have - want) <= bound)


def test_a_drafted_tree_over_the_bf16_cache(ext):
    """tree attention, verification and the move of the nodes that stand, one after the other: the
    verification's src and counts are what the move takes."""
    from cache_ops import paged
    lens, n, vocab = [60, 9], 7, 300
    k, v, table, _ = paged([x + n for x in lens], HKV, D, PAGE, seed=1)
    kc, vc = k.cuda(), v.cuda()
    g = torch.Generator().manual_seed(2)
    parents = torch.tensor([-1, 0, 0, 1, 1, 2, 3] * 2).int()
    q, prefix = torch.randn(2 * n, HQ, D, generator=g).bfloat16(), i32(lens)
    out, _ = ext.attn_sink_tree_paged(q.cuda(), kc, vc, table.cuda(), cu([n, n]).cuda(), prefix + n, parents.cuda(), n, 100)
    p = (out.float().flatten(1) @ torch.randn(HQ * D, vocab, generator=g).cuda()).softmax(-1)
    tok = p.argmax(-1).cpu()  # the likeliest token after each node, for its first child; another for the second
    chosen = torch.tensor([0 if q_ < 0 else int(tok[b * n + q_]) if q_ * 2 + 1 == i or q_ == 3 else 7
                           for b in range(2) for i, q_ in enumerate(parents[:n].tolist())]).int()
    u, un = torch.rand(2 * n, generator=g) * 0.2, torch.rand(2, generator=g)
    src, cnt, following = ext.attn_sink_verify_draft(p, chosen.cuda(), parents.cuda(), cu([n, n]).cuda(), u.cuda(), un.cuda(), n, base=prefix)
    ext.attn_sink_kv_compact(kc, vc, table.cuda(), src, cnt, base=prefix)
    assert ext.device_status() == 0 and int(cnt.max()) > 1
    for b, m in enumerate(lens):
        rows = slice(b * n, (b + 1) * n)
        path, token, _ = so.verify(co.to_np(p[rows]), None, chosen[rows].tolist(), parents[rows].tolist(), u[rows].tolist(), float(un[b]))
        assert int(following[b]) == token and int(cnt[b]) == len(path)
        for c, full in ((kc, k), (vc, v)):
            was, now = (co.tokens(x.cpu(), table[b], m + n) for x in (full, c))
            np.testing.assert_array_equal(now[:m], was[:m])
            np.testing.assert_array_equal(now[m:m + len(path)], was[[m + i for i in path]])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_parallel_samples(ext, fmt):
    """One prompt, four samples that share its pages; each goes its own way, some take over others'
    rows, the pool is brought together in between: every sample sees what it alone would have."""
    s, lone = Server(ext, 1, fmt), [Server(ext, 1, fmt) for _ in range(4)]
    k, v = s.normal(21, HKV, D), s.normal(21, HKV, D)
    for x in [s] + lone:
        x.grow(i32([21]))
        x.append(k, v, [21])
    s.table, s.lens = ext.attn_sink_pages_fork(s.table, s.refs, s.lens, i32([0, 0, 0, 0]), PAGE)
    for step in range(14):
        if step % 4 == 3:
            src = [[1, 1, 2, 0], [3, 0, 0, 2], [0, 1, 2, 2]][step // 4]
            s.table, s.lens = ext.attn_sink_pages_fork(s.table, s.refs, s.lens, i32(src), PAGE)
            old = lone
            lone = [Server(ext, 1, fmt) for _ in range(4)]
            for x, b in zip(lone, src):
                x.cache, x.table, x.refs, x.lens = ([t.clone() for t in old[b].cache], old[b].table.clone(), old[b].refs.clone(), old[b].lens)
        assert int(s.grow(s.lens + 1)) == 0
        k, v, q = s.normal(4, HKV, D), s.normal(4, HKV, D), s.normal(4, HQ, D)
        s.append(k, v, [1] * 4)
        if step % 5 == 2:
            held = int(ext.attn_sink_pages_compact(s.cache, s.table, s.refs, s.lens, PAGE))
            assert int((s.refs > 0).sum()) == held and not s.refs[held:].any()
        out, lse = ext.attn_sink_decode_paged_q8(q, *s.cache, s.table, s.lens)
        s.counts_agree()
        for b, x in enumerate(lone):
            x.grow(x.lens + 1)
            x.append(k[b:b + 1], v[b:b + 1], [1])
            o, z = ext.attn_sink_decode_paged_q8(q[b:b + 1], *x.cache, x.table, x.lens)
            assert same(o[0], out[b]) and same(z[0], lse[b])
    assert ext.device_status() == 0


def test_a_step_in_a_graph(ext):
    """Release, fork, reserve, append, extend, verify captured once and replayed: as the eager calls, on the
    state that each replay finds."""
    def make():
        s = Server(ext, 4, "e4m3", seed=5)
        s.grow(i32([33, 20, 17, 9]))
        s.append(s.normal(79, HKV, D), s.normal(79, HKV, D), [33, 20, 17, 9])
        return s
    n, vocab = 3, 200
    g = torch.Generator(device="cuda").manual_seed(9)
    k, v = (torch.randn(4 * n, HKV, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(4 * n, HQ, D, generator=g, device="cuda").bfloat16()
    head = torch.randn(HQ * D, vocab, generator=g, device="cuda")
    src, c = i32([1, 1, 0, 3]), cu([n] * 4).cuda()
    u, un = torch.rand(4 * n, generator=g, device="cuda"), torch.rand(4, generator=g, device="cuda")
    tok = torch.randint(0, vocab, (4 * n,), generator=g, device="cuda").int()

    def step(s, table, lens, stream=None):
        """One step on state held in place: table, lens, refs and caches."""
        kw = dict(stream=stream)
        t, l = ext.attn_sink_pages_fork(table, s.refs, lens, src, PAGE, **kw)
        new = l + n
        miss = ext.attn_sink_pages_reserve(s.cache, t, s.refs, l, new, PAGE, **kw)
        ext.attn_sink_kv_append_q8(k, v, *s.cache, t, new, cu_new=c, max_new=n, **kw)
        out, lse = ext.attn_sink_fwd_paged_q8(q, *s.cache, t, c, new, n, WIDTH * PAGE, **kw)
        o2, l2 = ext.attn_sink_decode_paged_q8(q[:4].contiguous(), *s.cache, t, new, **kw)
        big, _ = ext.attn_sink_fwd_paged_q8(q, *s.cache, t, c, new, 100, WIDTH * PAGE, **kw)  # the expanding path
        p = (out.float().flatten(1) @ head).softmax(-1)
        a, cnt, nxt = ext.attn_sink_verify_draft(p, tok, None, c, u, un, n, base=l, **kw)
        ext.attn_sink_pages_release(t, s.refs, new, l + cnt, PAGE, **kw)
        lens.copy_(l + cnt)
        table.copy_(t)
        held = ext.attn_sink_pages_compact(s.cache, table, s.refs, lens, PAGE, **kw)
        return [miss, out, lse, o2, l2, big, a, cnt, nxt, held]

    eager, graphed = make(), make()
    results = []
    for _ in range(3):
        results.append([t.clone() for t in step(eager, eager.table, eager.lens)])
    table, lens = graphed.table, graphed.lens
    keep = [t.clone() for t in (table, lens, graphed.refs, *graphed.cache)]
    step(graphed, table, lens)  # warm-up, undone
    for t, old in zip((table, lens, graphed.refs, *graphed.cache), keep):
        t.view(torch.uint8).copy_(old.view(torch.uint8))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(graphed, table, lens)
    for want in results:
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b) or same(a, b)
    for a, b in ((table, eager.table), (lens, eager.lens), (graphed.refs, eager.refs), *zip(graphed.cache, eager.cache)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert ext.device_status() == 0


NAMES = ("append", "decode", "few", "many", "verify", "fork", "reserve", "release", "compact", "copy")


def one_call(ext, name, seed):
    s = Server(ext, 2, "int8", seed)
    s.grow(i32([100, 37]))
    s.append(s.normal(137, HKV, D), s.normal(137, HKV, D), [100, 37])
    q, kn = s.normal(80, HQ, D), s.normal(80, HKV, D)
    c = cu([50, 30]).cuda()
    p = s.normal(80, 999).float().softmax(-1)
    tok, u, un = torch.randint(0, 999, (80,), generator=s.g, device="cuda").int(), torch.rand(80, generator=s.g, device="cuda"), torch.rand(2, device="cuda", generator=s.g)
    more, less, src = s.lens + 40, s.lens - 30, i32([1, 0])
    a, b, few = i32([1, 2]), i32([60, 61]), cu([5, 6]).cuda()
    table, refs, lens, cache = s.table, s.refs, s.lens, s.cache
    calls = dict(
        append=lambda st: ext.attn_sink_kv_append_q8(kn, kn, *cache, table, lens, cu_new=c, max_new=50, stream=st)[:0],
        decode=lambda st: ext.attn_sink_decode_paged_q8(q[:2], *cache, table, lens, stream=st),
        few=lambda st: ext.attn_sink_fwd_paged_q8(q[:11], *cache, table, few, lens, 6, 100, stream=st),
        many=lambda st: ext.attn_sink_fwd_paged_q8(q, *cache, table, c, lens, 50, 100, stream=st),
        verify=lambda st: ext.attn_sink_verify_draft(p, tok, None, c, u, un, 50, stream=st),
        fork=lambda st: ext.attn_sink_pages_fork(table, refs, lens, src, PAGE, stream=st),
        reserve=lambda st: (ext.attn_sink_pages_reserve(cache, table, refs, lens, more, PAGE, stream=st),),
        release=lambda st: ext.attn_sink_pages_release(table, refs, lens, less, PAGE, stream=st) or (),
        compact=lambda st: (ext.attn_sink_pages_compact(cache, table, refs, lens, PAGE, stream=st),),
        copy=lambda st: ext.attn_sink_pages_copy(cache, a, b, stream=st) or ())
    return calls[name], (table, refs, *cache)


@pytest.mark.parametrize("name", NAMES)
def test_dropped_outputs_on_another_stream(ext, name):
    """While the stream is still busy, tensors that the caller makes behind the call get other memory,
    and the call's effect is that of the same call on the current stream."""
    call, state = one_call(ext, name, 1)
    before = [t.clone() for t in state]
    shapes = [(t.shape, t.dtype) for t in call(None)]
    want = [t.clone() for t in state]
    for t, b in zip(state, before):
        t.view(torch.uint8).copy_(b.view(torch.uint8))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    call(side)
    mine = [torch.full(sh, 5, dtype=t, device="cuda") for sh, t in shapes for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.all(m == 5) for m in mine)
    for t, w in zip(state, want):
        assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("name", NAMES)
def test_a_forked_stream_inside_a_capture(ext, name):
    call, state = one_call(ext, name, 2)
    before = [t.clone() for t in state]
    keep = lambda ts: [t.clone() for t in ts]
    want = keep(call(None)) + keep(state)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = list(call(side))
        torch.cuda.current_stream().wait_stream(side)
        got = [t.clone() for t in got]
    for _ in range(2):
        for t, b in zip(state, before):
            t.view(torch.uint8).copy_(b.view(torch.uint8))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got + list(state), want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("name", NAMES)
def test_calls_on_two_streams_at_once(ext, name):
    """Calls that run side by side share nothing: each has the outputs and effects that it has alone."""
    made = [one_call(ext, name, seed) for seed in (5, 6)]
    before = [[t.clone() for t in state] for _, state in made]
    want = []
    for call, state in made:
        want.append([t.clone() for t in call(None)] + [t.clone() for t in state])
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(10):
        for (_, state), old in zip(made, before):
            for t, b in zip(state, old):
                t.view(torch.uint8).copy_(b.view(torch.uint8))
        torch.cuda.synchronize()
        got = []
        for (call, state), st in zip(made, streams):
            with torch.cuda.stream(st):
                torch.cuda._sleep(200_000)
            got.append((call(st), state))
        torch.cuda.synchronize()
        for (out, state), w in zip(got, want):
            for a, b in zip(list(out) + list(state), w):
                assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
    assert ext.device_status() == 0


def test_two_graphs_replayed_side_by_side(ext):
    """Graphs that were captured from the same calls have scratch of their own."""
    made = [one_call(ext, name, seed) for seed, name in enumerate(("many", "decode", "reserve", "few"), 7)]
    want = [[t.clone() for t in call(None)] for call, _ in made]
    before = [[t.clone() for t in state] for _, state in made]
    graphs = []
    for (call, state), old in zip(made, before):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(None)
        graphs.append((g, out))
    # (reserve gives pages once: what it finds the second time needs none)
    for (_, state), old in zip(made, before):
        for t, b in zip(state, old):
            t.view(torch.uint8).copy_(b.view(torch.uint8))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (_, out), w in zip(graphs, want):
        for a, b in zip(out, w):
            assert torch.equal(a, b) or same(a, b)
