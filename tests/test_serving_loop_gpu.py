"""The cache operators together, as a server runs them: a rotated prompt appended to
the paged cache, decode steps that keep the attention weights, evictions, and a
drafted tree that is checked, accepted along a path and compacted.

Every attention output is compared with the fp64 definition over the tokens that the
cache should hold, kept here as a list per request and KV head; tolerances as in
test_tree_gpu.py and test_rope_gpu.py."""
import numpy as np
import pytest
import torch

from oracle import cache_ops_oracle as co
from cache_ops import cu

pytestmark = pytest.mark.gpu

HQ, HKV, D, PAGE = 8, 2, 64, 16
GROUP = HQ // HKV


@pytest.fixture(scope="module")
def ext():
    from paged_kv_sink_gb300 import build
    build.build()
    import paged_kv_sink_gb300 as ext
    return ext


class Server:
    """Device state, and beside it what each request's cache should hold."""

    def __init__(self, ext, batch, tokens, seed):
        self.ext, self.batch = ext, batch
        self.g = torch.Generator().manual_seed(seed)
        per = -(-tokens // PAGE)
        perm = torch.randperm(batch * per, generator=self.g).int()
        self.table = perm.view(batch, per).cuda().contiguous()
        self.k, self.v = (torch.full((batch * per, PAGE, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                          for _ in range(2))
        self.weights = torch.zeros(batch, HKV, per * PAGE, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.seen = [0] * batch                       # positions used so far, evicted ones too
        self.keys = [[[] for _ in range(HKV)] for _ in range(batch)]    # exact (key, value) rows per head
        self.sink = (torch.rand(HQ, generator=self.g) * 3 - 1).cuda()
        self.freqs, self.scale = ext.attn_sink_rope_freqs(32, scaling="yarn", factor=4.0, original_len=64)

    def rows(self, n, heads):
        return torch.randn(n, heads, D, generator=self.g).bfloat16()

    def append(self, new, positions=None):
        """Appends new[b] tokens to every request; returns the rotated queries."""
        T = sum(new)
        q, k, v = self.rows(T, HQ), self.rows(T, HKV), self.rows(T, HKV)
        if positions is None:
            positions = torch.cat([torch.arange(s, s + n) for s, n in zip(self.seen, new)]).int()
        self.lens += torch.tensor(new, dtype=torch.int32, device="cuda")
        out = self.ext.attn_sink_rope_kv_append(q.cuda(), k.cuda(), v.cuda(), self.k, self.v, self.table, self.lens,
                                                self.freqs, cu_new=cu(new).cuda(), max_new=max(new),
                                                positions=positions.cuda(), attn_scale=self.scale)
        # what the cache holds is the rotated key rounded to bf16: checked, then taken from there
        exact = co.rotate(k, positions, self.freqs, False, self.scale)
        row = 0
        for b, n in enumerate(new):
            length = int(self.lens[b])
            held = self.tokens(b, length)
            for i in range(n):
                at = length - n + i
                err = np.abs(held[0][at] - exact[row])
                assert np.all(err <= 2.0 ** -8 * np.abs(exact[row]) + 2.0 ** -19 * 10)
                assert np.array_equal(held[1][at], co.to_np(v[row]))
                for h in range(HKV):
                    self.keys[b][h].append((held[0][at, h], held[1][at, h]))
                row += 1
        return out

    def tokens(self, b, n):
        return [co.tokens(c.cpu(), self.table[b].cpu(), n) for c in (self.k, self.v)]

    def check(self, q, out, lse, b, seen=None):
        """out (n, HQ, D), lse (HQ, n) of request b's rows q against the lists."""
        probs = []
        for h in range(HKV):
            k, v = (np.stack([t[i] for t in self.keys[b][h]])[:, None] for i in range(2))
            hs = slice(h * GROUP, (h + 1) * GROUP)
            vis = np.ones((q.shape[0], k.shape[0]), bool) if seen is None else seen
            O, L, P, A = co.attend(q[:, hs], k, v, vis, self.sink[hs].cpu().numpy(), D ** -0.5)
            err = np.abs(co.to_np(out[:, hs]) - O)
            assert np.all(err <= 2.0 ** -8 * (A + np.abs(O)) + 2.0 ** -13 * A)
            np.testing.assert_allclose(lse[hs].cpu().numpy(), L, atol=1.5e-4)
            probs.append(P[:, 0].sum(0))
        return probs


def test_prompt_decode_evict_draft_accept(ext):
    s = Server(ext, 2, 400, seed=3)
    prompt = [150, 40]
    q = s.append(prompt)
    out, lse = ext.attn_sink_fwd_paged(q, s.k, s.v, s.table, cu(prompt).cuda(), s.lens, 150, 150, sink=s.sink)
    for b, (r0, n) in enumerate(((0, 150), (150, 40))):
        s.check(q[r0:r0 + n].cpu(), out[r0:r0 + n], lse[:, r0:r0 + n], b, np.tril(np.ones((n, n), bool)))
    s.seen = list(prompt)
    want_w = [[np.zeros(len(s.keys[b][h])) for h in range(HKV)] for b in range(2)]

    for step in range(6):
        # one token each, with its weights kept
        q = s.append([1, 1])
        out, lse = ext.attn_sink_decode_paged_weights(q, s.k, s.v, s.table, s.lens, s.weights, s.sink)
        for b in range(2):
            s.seen[b] += 1
            probs = s.check(q[b:b + 1].cpu(), out[b:b + 1], lse[b][:, None], b)
            for h in range(HKV):
                want_w[b][h] = np.append(want_w[b][h], 0.0) + probs[h]
                got = s.weights[b, h].cpu().numpy()
                n = len(want_w[b][h])
                assert np.all(np.abs(got[:n] - want_w[b][h]) <= 4e-4 * want_w[b][h] + 1e-7) and not got[n:].any()
        if step in (2, 4):
            # down to 100 tokens: request 1 (below that) keeps everything
            before = s.weights.cpu()
            new, kept = ext.attn_sink_evict_paged(s.k, s.v, s.table, s.lens, s.weights, 100, keep_first=4, keep_last=16)
            for b in range(2):
                n = int(s.lens[b])
                for h in range(HKV):
                    src = co.evict(before[b, h].numpy(), n, 100, 4, 16)
                    assert kept[b, h, :len(src)].tolist() == src.tolist()
                    s.keys[b][h] = [s.keys[b][h][t] for t in src]
                    want_w[b][h] = want_w[b][h][src]
                held = s.tokens(b, int(new[b]))
                for h in range(HKV):
                    assert np.array_equal(held[0][:, h], np.stack([t[0] for t in s.keys[b][h]]))
                    assert np.array_equal(held[1][:, h], np.stack([t[1] for t in s.keys[b][h]]))
            s.lens = new

    # a draft of 12 and 5 nodes; positions go on from the prefix by depth
    nodes = [12, 5]
    parents = [-1, 0, 0, 1, 3, -1, 5, 4, 7, 8, 2, 9] + [-1, 0, 1, 2, 0]
    depth = [0, 1, 1, 2, 3, 0, 1, 4, 5, 6, 2, 7] + [0, 1, 2, 3, 1]
    prefix = s.lens.clone()
    start = [s.seen[0]] * 12 + [s.seen[1]] * 5
    q = s.append(nodes, torch.tensor([a + d for a, d in zip(start, depth)]).int())
    out, lse = ext.attn_sink_tree_paged(q, s.k, s.v, s.table, cu(nodes).cuda(), s.lens, torch.tensor(parents).int().cuda(),
                                        12, 120, sink=s.sink)
    for b, (r0, n) in enumerate(((0, 12), (12, 5))):
        seen = co.tree_seen(parents[r0:r0 + n], int(prefix[b]))
        s.check(q[r0:r0 + n].cpu(), out[r0:r0 + n], lse[:, r0:r0 + n], b, seen)

    # accept 0-1-3-4-7 and nothing but node 0
    paths = [[0, 1, 3, 4, 7], [0]]
    counts = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
    src = torch.zeros(2, 5, dtype=torch.int32)
    for b, p in enumerate(paths):
        src[b, :len(p)] = int(prefix[b]) + torch.tensor(p)
    ext.attn_sink_kv_compact(s.k, s.v, s.table, src.cuda(), counts, base=prefix)
    s.lens = prefix + counts
    for b, p in enumerate(paths):
        n = int(prefix[b])
        for h in range(HKV):
            s.keys[b][h] = s.keys[b][h][:n] + [s.keys[b][h][n + i] for i in p]
        s.seen[b] += len(p)
    # and decode goes on as if the accepted tokens had come one by one
    q = s.append([1, 1])
    out, lse = ext.attn_sink_decode_paged(q, s.k, s.v, s.table, s.lens, s.sink)
    for b in range(2):
        s.check(q[b:b + 1].cpu(), out[b:b + 1], lse[b][:, None], b)
    torch.cuda.synchronize()
    assert ext.device_status() == 0


def test_training_step_with_rotary_positions(ext):
    """Rotation, attention with a learnable sink and their gradients in one graph: the
    gradient of q equals the attention's own, rotated back."""
    g = torch.Generator().manual_seed(5)
    T = 96
    q, k, v = (torch.randn(T, h, D, generator=g).bfloat16().cuda().requires_grad_() for h in (HQ, HKV, HKV))
    sink = torch.zeros(HQ, device="cuda", requires_grad=True)
    dout = torch.randn(T, HQ, D, generator=g).bfloat16().cuda()
    pos = torch.cat([torch.arange(64), torch.arange(32)]).int().cuda()
    c = cu([64, 32]).cuda()
    f, m = ext.attn_sink_rope_freqs(D)
    yq, yk = ext.attn_sink_rope_func(q, k, pos, f, attn_scale=m)
    out = ext.attn_sink_varlen_func(yq, yk, v, c, c, 64, 64, learnable_sink=sink)
    gq, gk, gs, gyq, gyk = torch.autograd.grad(out, (q, k, sink, yq, yk), dout)
    for got, inner in ((gq, gyq), (gk, gyk)):
        want = co.rotate(inner, pos, f, False, m, inverse=True)
        size = np.abs(co.to_np(inner))
        pair = np.concatenate([size[..., :32] + size[..., 32:]] * 2, -1)
        assert np.all(np.abs(co.to_np(got) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * pair)
    assert torch.all(torch.isfinite(gs)) and gs.abs().max() > 0


def test_caches_whose_offsets_pass_32_bits(ext):
    """The same calls on a small cache and on the same pages at the end of one of 2.4e9
    elements give the same bits."""
    from cache_ops import paged, same
    k, v, table, sl = paged([700, 90], 8, 64, 16, seed=31)
    pool, far = k.shape[0], 290000
    g = torch.Generator().manual_seed(32)
    q, nk, nv = (torch.randn(8, h, 64, generator=g).bfloat16().cuda() for h in (64, 8, 8))
    cu_new, parents = cu([5, 3]).cuda(), torch.tensor([-1, 0, 0, 1, -1, -1, 0, 1]).int().cuda()
    freqs, _ = ext.attn_sink_rope_freqs(64)
    got = []
    for at in (0, far):
        kc, vc = (torch.empty(at + pool, 16, 8, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        kc[at:], vc[at:] = k.cuda(), v.cuda()
        tc, n = (table + at * (table >= 0).int()).cuda(), sl.cuda()
        qr = ext.attn_sink_rope_kv_append(q, nk, nv, kc, vc, tc, n, freqs, cu_new=cu_new, max_new=5)
        out, lse = ext.attn_sink_tree_paged(qr, kc, vc, tc, cu_new, n, parents, 5, 700)
        keep = torch.tensor([[0, 2, 4], [1, 2, 0]]).int().cuda() + (n - torch.tensor([5, 3], device="cuda").int())[:, None]
        counts = torch.tensor([3, 2]).int().cuda()
        ext.attn_sink_kv_compact(kc, vc, tc, keep, counts, base=n - torch.tensor([5, 3]).int().cuda())
        n = n - torch.tensor([2, 1]).int().cuda()
        w = torch.zeros(2, 8, 700, device="cuda")
        out2, lse2 = ext.attn_sink_decode_paged_weights(q[:2], kc, vc, tc, n, w)
        new, kept = ext.attn_sink_evict_paged(kc, vc, tc, n, w, 80, keep_first=4, keep_last=8)
        torch.cuda.synchronize()
        assert ext.device_status() == 0
        got.append([t.cpu() for t in (qr, out, lse, out2, lse2, w, new, kept, kc[at:], vc[at:])])
        del kc, vc
        torch.cuda.empty_cache()
    for a, b in zip(*got):
        assert torch.equal(a, b) if a.dtype == torch.int32 else same(a, b)


def test_a_captured_loop_equals_the_eager_one(ext):
    """A decode step with its weights, an eviction, a draft and the move of its accepted path,
    captured in one CUDA graph, give the eager calls' bits on every replay."""
    from cache_ops import same
    sl = torch.tensor([180, 95]).int()
    table = torch.randperm(32, generator=torch.Generator().manual_seed(51)).int().view(2, 16)
    g = torch.Generator().manual_seed(52)
    k, v = (torch.randn(32, PAGE, HKV, D, generator=g).bfloat16() for _ in range(2))
    T = [1, 1], [6, 3]
    parents = torch.tensor([-1, 0, 0, 1, 3, -1] + [-1, 0, 1]).int().cuda()
    depth = torch.tensor([0, 1, 1, 2, 3, 0] + [0, 1, 2]).int().cuda()
    owner = torch.tensor([0] * 6 + [1] * 3).cuda()
    path = torch.tensor([[0, 1, 3], [0, 1, 0]]).int().cuda()
    accepted, drafted = torch.tensor([3, 2]).int().cuda(), torch.tensor([6, 3]).int().cuda()
    table, c2 = table.cuda(), cu(T[1]).cuda()
    f, m = ext.attn_sink_rope_freqs(D, scaling="bands", factor=4.0, original_len=128)
    sink = torch.linspace(-1, 2, HQ).cuda()
    kc, vc, lens = k.cuda(), v.cuda(), sl.cuda()
    w = torch.zeros(2, HKV, table.shape[1] * PAGE, device="cuda")
    rows = [torch.empty(sum(n), h, D, dtype=torch.bfloat16, device="cuda") for n in T for h in (HQ, HKV, HKV)]

    def reset(seed):
        g = torch.Generator().manual_seed(seed)
        kc.copy_(k), vc.copy_(v), lens.copy_(sl), w.zero_()
        for r in rows:
            r.copy_(torch.randn(r.shape, generator=g))

    def step():
        lens.add_(1)
        q = ext.attn_sink_rope_kv_append(*rows[:3], kc, vc, table, lens, f, attn_scale=m)
        out, lse = ext.attn_sink_decode_paged_weights(q, kc, vc, table, lens, w, sink, 4, 100)
        new, kept = ext.attn_sink_evict_paged(kc, vc, table, lens, w, 96, keep_first=4, keep_last=32)
        n = new + drafted
        pos = new[owner] + depth
        q2 = ext.attn_sink_rope_kv_append(*rows[3:], kc, vc, table, n, f, cu_new=c2, max_new=6, positions=pos, attn_scale=m)
        out2, lse2 = ext.attn_sink_tree_paged(q2, kc, vc, table, c2, n, parents, 6, 110, sink=sink)
        ext.attn_sink_kv_compact(kc, vc, table, new[:, None] + path, accepted, base=new)
        after = new + accepted
        out3, lse3 = ext.attn_sink_decode_paged(q, kc, vc, table, after, sink)
        return [q, out, lse, new, kept, q2, out2, lse2, after, out3, lse3]

    want = []
    for seed in (1, 2):
        reset(seed)
        want.append([t.clone() for t in step() + [kc, vc, w]])
    torch.cuda.synchronize()
    assert not same(want[0][1], want[1][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (2, 1, 2):
        reset(seed)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got + [kc, vc, w], want[seed - 1]):
            assert torch.equal(a, b) if a.dtype == torch.int32 else same(a, b)
    assert ext.device_status() == 0
