"""Pages' bookkeeping against the model in whole numbers: tables, counts, lengths and the pages'
contents after every call."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ext():
    from paged_kv_sink_gb300 import build
    build.build()
    import paged_kv_sink_gb300 as ext
    return ext


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Both:
    """The model and the device's state, side by side."""

    def __init__(self, ext, lens, page, pool, width, seed=0, kinds=("bf16",)):
        g = np.random.default_rng(seed)
        n = [-(-t // page) for t in lens]
        perm = g.permutation(pool)
        table, at = np.full((len(lens), width), -1), 0
        for b, m in enumerate(n):
            table[b, :m] = perm[at:at + m]
            at += m
        refs = np.zeros(pool, int)
        refs[table[table >= 0]] = 1
        self.ext, self.page = ext, page
        self.m = so.Pages(table, refs, lens, page, np.arange(pool))
        self.table, self.refs, self.lens = i32(table), i32(refs), i32(lens)
        make = dict(bf16=lambda: torch.randn(pool, page, 2, 64).bfloat16(), bytes=lambda: torch.randint(0, 255, (pool, 13)).to(torch.uint8),
                    scales=lambda: torch.rand(pool, 1, 3), big=lambda: torch.randn(pool, page, 4, 128).bfloat16())
        torch.manual_seed(seed)
        self.start = [make[k]() for k in kinds]
        self.caches = [t.cuda() for t in self.start]

    def same(self):
        np.testing.assert_array_equal(self.table.cpu().numpy(), self.m.table)
        np.testing.assert_array_equal(self.refs.cpu().numpy(), self.m.refs)
        np.testing.assert_array_equal(self.lens.cpu().numpy(), self.m.lens)
        used = np.flatnonzero(self.m.refs > 0)
        for c, s in zip(self.caches, self.start):
            assert torch.equal(c[torch.from_numpy(used).cuda()].cpu(), s[torch.from_numpy(self.m.labels[used])])
        held = np.zeros(len(self.m.refs), int)
        for b, n in enumerate(self.m.lens):
            np.add.at(held, self.m.table[b, :self.m.held(n)], 1)
        np.testing.assert_array_equal(held, self.m.refs)

    def fork(self, src):
        self.table, self.lens = self.ext.attn_sink_pages_fork(self.table, self.refs, self.lens, i32(src), self.page)
        self.m.fork(src)

    def release(self, new):
        self.ext.attn_sink_pages_release(self.table, self.refs, self.lens, i32(new), self.page)
        self.lens = i32(new)
        self.m.release(new)

    def reserve(self, new):
        short = self.m.reserve(new)
        got = int(self.ext.attn_sink_pages_reserve(self.caches, self.table, self.refs, self.lens, i32(new), self.page))
        assert got == short
        if not short:
            self.lens = i32(new)
        return short

    def compact(self):
        held = self.m.compact()
        assert int(self.ext.attn_sink_pages_compact(self.caches, self.table, self.refs, self.lens, self.page)) == held


@pytest.mark.parametrize("page,pool,rows,kinds", [(16, 200, 6, ("bf16",)), (1, 300, 5, ("bytes",)), (7, 97, 9, ("bf16", "bytes", "scales")),
                                                  (64, 5000, 40, ("bf16", "bf16", "scales", "scales")), (8, 40000, 1500, ("scales",))])
def test_random_calls(ext, page, pool, rows, kinds):
    """Forks (more rows, fewer, none of some), growth with shared last pages, shrinking, compaction."""
    g = np.random.default_rng(pool)
    cap = max(2 * page, pool * page // (3 * rows))
    width = cap // page + 3
    s = Both(ext, g.integers(0, cap // 2, rows).tolist(), page, pool, width, seed=pool, kinds=kinds)
    s.same()
    for step in range(8):
        n = rows if step % 3 else max(1, rows + int(g.integers(-rows // 2, rows // 3)))
        src = g.integers(-1, len(s.m.lens), n)
        src[g.random(n) < 0.3] = int(g.integers(0, len(s.m.lens)))
        s.fork(src.tolist())
        s.same()
        s.reserve((s.m.lens + g.integers(0, cap // 6 + 2, n)).clip(max=width * page).tolist())
        s.same()
        s.release((s.m.lens * g.random(n) * (g.random(n) < 0.8)).astype(int).tolist())
        s.same()
        if step % 2:
            s.compact()
            s.same()
    assert ext.device_status() & ~ext._lib.DEV_POOL == 0  # some growth may have been refused


def test_all_holders_grow_the_last_keeps_the_page(ext):
    s = Both(ext, [20, 33, 16], 16, 40, 8, kinds=("big", "bytes"))
    s.fork([0, 0, 1, 0, 2, 1, -1, 0])
    s.reserve([21, 36, 40, 20, 17, 33, 1, 22])   # rows 3 and 5 do not grow: row 3 and the others share on
    s.same()
    s.fork([0, 0, 0])
    assert s.reserve([22, 22, 22]) == 0          # all holders: rows 0 and 1 copy, row 2 keeps
    assert s.m.table[2, 1] not in (s.m.table[0, 1], s.m.table[1, 1])
    s.same()
    assert ext.device_status() == 0


def test_too_few_pages_change_nothing(ext):
    s = Both(ext, [20, 20], 16, 6, 8)
    assert s.reserve([64, 33]) == 1
    s.same()
    assert ext.device_status() == ext._lib.DEV_POOL
    assert s.reserve([48, 33]) == 0
    s.same()
    assert s.reserve([48, 33]) == 0 and s.reserve([49, 33]) == 1
    ext.device_status()


def test_full_and_empty_pools_compact(ext):
    for lens, pool in (([64, 64], 8), ([0, 0], 8), ([1], 1), ([16 * 5], 4096)):
        s = Both(ext, lens, 16, pool, 8, seed=pool)
        s.compact()
        s.same()
        s.compact()
        s.same()
    assert ext.device_status() == 0


def test_a_pool_of_many_pages(ext):
    s = Both(ext, [3000, 17, 40000], 1, 300000, 70000, kinds=("scales",))
    s.compact()
    s.same()
    s.reserve([3001, 20000, 69999])
    s.same()
    s.release([0, 19000, 5])
    s.compact()
    s.same()
    assert ext.device_status() == 0


@pytest.mark.parametrize("pool,rows,skew", [(600000, 3, 0), (700001, 3, 1), (20000, 9000, 0), (3000, 70, 3)])
def test_more_pages_and_requests_than_threads_hold(ext, pool, rows, skew):
    """Pools above 524288 pages, more requests than the cluster has threads, counts off a 16-byte border."""
    g = np.random.default_rng(pool)
    top = pool // (3 * rows)
    s = Both(ext, g.integers(0, top + 1, rows).tolist(), 1, pool, top + 2, seed=1, kinds=("scales",))
    refs = torch.zeros(pool + skew, dtype=torch.int32, device="cuda")[skew:]
    s.refs = refs.copy_(s.refs)
    s.compact()
    s.same()
    s.reserve((s.m.lens + g.integers(0, 3, rows)).clip(max=top + 2).tolist())
    s.same()
    s.release((s.m.lens // 2).tolist())
    s.fork(g.integers(0, rows, rows).tolist())
    s.reserve((s.m.lens + 1).tolist())
    s.same()
    s.compact()
    s.same()
    assert ext.device_status() == 0


def test_copies(ext):
    for shape, dtype in (((9, 13), torch.uint8), ((9, 16, 2, 64), torch.bfloat16), ((9, 3), torch.float32), ((9, 70001), torch.int16),
                         ((9, 1 << 18), torch.float32)):
        x = torch.randint(-100, 100, shape).to(dtype)
        y = x.cuda()
        z = torch.arange(9.0).view(9, 1).cuda()
        ext.attn_sink_pages_copy([y, z], i32([0, 4, -1, 7, 5]), i32([8, 3, -1, 1, 5]))
        x[[8, 3, 1]] = x[[0, 4, 7]]
        assert torch.equal(y.cpu(), x) and z.flatten().tolist() == [0, 7, 2, 4, 4, 5, 6, 7, 0]
    assert ext.device_status() == 0
    flat = torch.arange(64, dtype=torch.uint8, device="cuda")[1:61].view(4, 15)  # no alignment at all
    ext.attn_sink_pages_copy(flat, i32([0]), i32([3]))
    assert torch.equal(flat[3], flat[0])
    before = y.clone()
    ext.attn_sink_pages_copy(y, i32([0, 9, -1]), i32([99, 1, 2]))
    assert torch.equal(before, y) and ext.device_status() == ext._lib.DEV_PAGE_OOB


def test_contradictions_are_reported(ext):
    D = ext._lib
    s = Both(ext, [40, 40], 16, 10, 4)
    ext.device_status()
    table, refs = s.table.clone(), s.refs.clone()
    ext.attn_sink_pages_release(table, refs, s.lens, i32([41, 65]), 16)   # growth; 65 tokens do not fit 4 pages
    assert torch.equal(table, s.table) and torch.equal(refs, s.refs)
    assert ext.device_status() == D.DEV_POOL | D.DEV_SEQLEN_OOB
    refs = torch.zeros_like(s.refs)
    ext.attn_sink_pages_release(table.clone(), refs, s.lens, i32([0, 0]), 16)  # held, but not counted
    assert torch.all(refs == 0) and ext.device_status() == D.DEV_POOL
    bad = s.table.clone()
    bad[0, 2], bad[1, 1] = 10, -3
    refs = s.refs.clone()
    ext.attn_sink_pages_fork(bad, refs, s.lens, i32([0, 5]), 16)
    assert ext.device_status() == D.DEV_PAGE_OOB | D.DEV_POOL
    refs, t = s.refs.clone(), bad.clone()
    assert int(ext.attn_sink_pages_reserve(s.caches, t, refs, s.lens, i32([39, 41]), 16)) == 0
    assert torch.equal(t, bad) and torch.equal(refs, s.refs) and ext.device_status() == D.DEV_POOL
    assert int(ext.attn_sink_pages_reserve(s.caches, t, refs, s.lens, i32([41, 999]), 16)) == 0
    assert torch.equal(t, bad) and ext.device_status() == D.DEV_PAGE_OOB | D.DEV_SEQLEN_OOB
    ext.attn_sink_pages_compact(s.caches, bad.clone(), refs, s.lens, 16)
    assert ext.device_status() == D.DEV_PAGE_OOB


def test_no_requests(ext):
    t, r, e = torch.zeros(0, 3, dtype=torch.int32, device="cuda"), i32([0, 0]), i32([])
    out, lens = ext.attn_sink_pages_fork(t, r, e, i32([-1, -1]), 4)
    assert out.tolist() == [[-1] * 3] * 2 and lens.tolist() == [0, 0]
    assert int(ext.attn_sink_pages_reserve([], t, r, e, e, 4)) == 0
    assert int(ext.attn_sink_pages_compact([], t, r, e, 4)) == 0
    ext.attn_sink_pages_release(t, r, e, e, 4)
    assert ext.device_status() == 0
