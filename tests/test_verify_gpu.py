"""Verification of drafted tokens against the definition in fp64.  Whole numbers: all must be equal.
The kernel's sums are exact in units of 2^-44, so that a drawn place would have to lie within
vocab 2^-44 of a border to differ; inputs are drawn with 24 random bits."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from cache_ops import cu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ext():
    from paged_kv_sink_gb300 import build
    build.build()
    import paged_kv_sink_gb300 as ext
    return ext


def case(nodes, vocab, arity, sampled, dtype, seed, near=0.5, sharp=3.0):
    """Random rows, trees in which up to `arity` nodes hang on one, tokens drawn from the draft."""
    g = torch.Generator().manual_seed(seed)
    rows = sum(nodes)
    x = torch.randn(rows, vocab, generator=g) * sharp
    target = x.softmax(-1).to(dtype)
    y = (x + near * torch.randn(rows, vocab, generator=g)).softmax(-1)
    parents, tokens, r0 = [], [], 0
    for n in nodes:
        for i in range(n):
            p = -1 if i == 0 else max(0, (i - 1) // arity)
            parents.append(p)
            tokens.append(int(torch.multinomial(y[r0 + max(p, 0)], 1, generator=g)))
        r0 += n
    return dict(target=target, draft=y.to(dtype) if sampled else None, tokens=torch.tensor(tokens, dtype=torch.int32),
                parents=torch.tensor(parents, dtype=torch.int32), cu=cu(nodes), u=torch.rand(rows, generator=g),
                u_next=torch.rand(len(nodes), generator=g), nodes=nodes)


def run(ext, c, base=None, most=None, **kw):
    d = lambda t: None if t is None else t.cuda()
    most = max(c["nodes"] + [0]) if most is None else most
    got = ext.attn_sink_verify_draft(d(c["target"]), d(c["tokens"]), d(c["parents"]), d(c["cu"]), d(c["u"]), d(c["u_next"]), most,
                                     draft=d(c["draft"]), base=d(base), **kw)
    return [t.cpu().numpy() for t in got]


def expect(c, b, most=256):
    r0, r1 = int(c["cu"][b]), int(c["cu"][b + 1])
    r1 = min(r1, r0 + most)
    par = [-1] + list(range(r1 - r0 - 1)) if c["parents"] is None else c["parents"][r0:r1].tolist()
    for i, p in enumerate(par):
        if i and not 0 <= p < i:
            par[i] = -9
    num = lambda t: t.double().numpy()
    return so.verify(num(c["target"][r0:r1]), None if c["draft"] is None else num(c["draft"][r0:r1]), c["tokens"][r0:r1].tolist(),
                     par, num(c["u"][r0:r1]), float(c["u_next"][b]))


def compare(ext, c, base=None, most=None):
    src, counts, following = run(ext, c, base, most)
    for b, n in enumerate(c["nodes"]):
        if n == 0:
            assert counts[b] == 0 and following[b] == -1 and np.all(src[b] == -1)
            continue
        path, token, _ = expect(c, b, src.shape[1])
        assert counts[b] == len(path) and following[b] == token, (b, path, token, counts[b], following[b])
        first = 0 if base is None else int(base[b])
        assert src[b, :len(path)].tolist() == [first + i for i in path] and np.all(src[b, len(path):] == -1)
    return counts


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("vocab,arity", [(1, 1), (2, 2), (31, 3), (1000, 1), (4096, 2), (4097, 3), (8191, 2), (33001, 4), (50000, 1)])
def test_matches_definition(ext, vocab, arity, sampled, dtype):
    nodes = [1, 2, 9, 0, 17, 33, 5, 12]
    c = case(nodes, vocab, arity, sampled, dtype, seed=vocab + arity)
    counts = compare(ext, c, base=torch.arange(8).int() * 1000)
    assert ext.device_status() == 0
    # (tokens drawn from a model near the target's are taken often, chosen ones with probability p(x))
    assert vocab < 4000 or not sampled or counts.max() > 1


@pytest.mark.parametrize("sampled", [True, False])
@pytest.mark.parametrize("vocab", [50, 40000])
def test_many_requests_and_chains(ext, vocab, sampled):
    nodes = [1 + b % 8 for b in range(300 if vocab == 50 else 60)]
    c = case(nodes, vocab, 1, sampled, torch.float32, seed=3, near=0.2, sharp=2.0)
    want = run(ext, c)
    c["parents"] = None  # a chain
    compare(ext, c)
    for a, b in zip(run(ext, c), want):
        np.testing.assert_array_equal(a, b)


@pytest.mark.parametrize("sampled", [True, False])
def test_256_nodes_on_one(ext, sampled):
    """A root with 255 children, the same tokens more than once, most of them refused."""
    c = case([256, 256], 600, 255, sampled, torch.float32, seed=5, near=1.5)
    c["u"][:] = 0.999999
    c["u"][300:] = 1.0 - 2.0 ** -24
    compare(ext, c)
    c["u"][:] = 0.9
    compare(ext, c)


def test_skewed_and_strided_rows(ext):
    """Rows at every alignment, the draft's unlike the target's; columns of a wider matrix."""
    for dtype in (torch.float32, torch.bfloat16):
        for at, bt in ((1, 1), (3, 2), (0, 5)):
            c = case([7, 9], 6001, 2, True, dtype, seed=at)
            wide = torch.full((16, 6020), 9.0, dtype=dtype).cuda()
            wide2 = torch.full((16, 6031), 9.0, dtype=dtype).cuda()
            p, q = wide[:, at:at + 6001], wide2[:, bt:bt + 6001]
            p.copy_(c["target"])
            q.copy_(c["draft"])
            got = ext.attn_sink_verify_draft(p, c["tokens"].cuda(), c["parents"].cuda(), c["cu"].cuda(), c["u"].cuda(),
                                             c["u_next"].cuda(), 9, draft=q)
            for a, b in zip(got, run(ext, c)):
                np.testing.assert_array_equal(a.cpu().numpy(), b)
            compare(ext, c)


def test_ends_of_the_random_numbers(ext):
    """u_next 0 gives the first token with any probability, just below 1 (and 1, above it) the
    last; NaN counts as 0."""
    p = torch.zeros(6, 5000)
    p[:, 17], p[:, 4000], p[:, 4321] = 0.25, 0.5, 0.25
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 7.0, float("nan"), 0.25])
    c = dict(target=p, draft=None, tokens=torch.zeros(6).int(), parents=None, cu=cu([1] * 6), u=torch.zeros(6), u_next=u, nodes=[1] * 6)
    assert run(ext, c)[2].tolist() == [17, 4321, 4321, 4321, 17, 4000]
    assert ext.device_status() == 0


def test_draft_equal_to_target_is_taken(ext):
    c = case([9, 9], 3000, 1, True, torch.float32, seed=8, near=0.0)
    c["u"][:] = 1 - 2.0 ** -24
    assert run(ext, c)[1].tolist() == [9, 9]
    compare(ext, c)


def test_nothing_left_and_nothing_there(ext):
    """A residual without mass: the target's row; a row without mass: -1 and a status bit; values
    that are no probabilities count as clamped."""
    p = torch.zeros(8, 300)
    q = torch.zeros(8, 300)
    p[0, 5] = 1.0                                       # request 0: p <= q everywhere, child refused (q > p at its token)
    q[0, 5], q[0, 6] = 1.0, 1.0
    p[3, 9], p[3, 8], p[3, 2] = float("nan"), -1.0, 2.0  # request 1: one token counts, as 1
    p[6, 250] = 1e-30                                   # request 2: no mass in units of 2^-44
    c = dict(target=p, draft=q, tokens=torch.tensor([0, 6, 0, 0, 8, 0, 0, 0]).int(), parents=None, cu=cu([2, 3, 3]),
             u=torch.full((8,), 0.5), u_next=torch.tensor([0.9, 0.99, 0.5]), nodes=[2, 3, 3])
    c["target"] = torch.cat([p[:2], p[3:4], p[4:6], p[6:7], p[:2] * 0])
    c["draft"] = torch.cat([q[:2], q[4:8], q[4:6]])
    ext.device_status()
    src, counts, following = run(ext, c)
    assert counts.tolist() == [1, 1, 1] and following.tolist() == [5, 2, -1]
    assert ext.device_status() == ext._lib.DEV_PROB


def test_bad_nodes_are_left_out(ext):
    """Parents out of range, tokens outside the vocabulary, more nodes than max_nodes or rows."""
    D = ext._lib
    c = case([6, 6], 500, 2, False, torch.float32, seed=4)
    c["u"][:] = 0.0
    c["parents"][3], c["parents"][8], c["parents"][9] = 3, -5, 77
    ext.device_status()
    compare(ext, c)
    assert ext.device_status() == D.DEV_TREE
    c = case([6, 6], 500, 2, False, torch.float32, seed=4)
    c["tokens"][1], c["tokens"][2], c["tokens"][7] = 500, -1, 2 ** 31 - 1
    compare(ext, c)
    assert ext.device_status() == D.DEV_PROB
    c = case([6, 3], 500, 1, False, torch.float32, seed=4)
    c["u"][:] = 0.0
    assert compare(ext, c, most=4).tolist() == [4, 3]
    assert ext.device_status() == D.DEV_SEQLEN_OOB
    c["cu"] = torch.tensor([0, 6, 11]).int()  # two rows more than there are
    src, counts, _ = run(ext, c)
    assert counts.tolist() == [6, 3] and ext.device_status() == D.DEV_SEQLEN_OOB


def test_no_requests_no_rows_no_nodes(ext):
    z = lambda *s: torch.zeros(*s, device="cuda")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    src, counts, following = ext.attn_sink_verify_draft(z(0, 40), i(0), None, i(1), z(0), z(0), 4)
    assert src.shape == (0, 4)
    src, counts, following = ext.attn_sink_verify_draft(z(0, 40), i(0), None, i(3), z(0), z(2), 0)
    assert counts.tolist() == [0, 0] and following.tolist() == [-1, -1] and src.shape == (2, 0)
    assert ext.device_status() == 0


def test_the_largest_vocabulary(ext):
    vocab = (1 << 20) - 1
    c = case([3], vocab, 2, True, torch.float32, seed=1)
    compare(ext, c)
    c = case([2, 2], vocab, 1, False, torch.bfloat16, seed=2)
    c["u"][:] = 1.0
    compare(ext, c)


def test_offsets_past_32_bits(ext):
    """Rows that start more than 2^32 bytes into the tensor."""
    rows, vocab = 4200, 524288
    p = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(1)
    small = torch.randn(3, vocab, generator=g).softmax(-1).bfloat16()
    p[-3:] = small.cuda()
    tok = torch.zeros(rows, dtype=torch.int32)
    tok[-2:] = torch.tensor([123, vocab - 1])
    c = torch.tensor([0, rows - 3, rows]).int()
    u = torch.zeros(rows)
    following = ext.attn_sink_verify_draft(p, tok.cuda(), None, c.cuda(), u.cuda(), torch.tensor([0.0, 0.7]).cuda(), 3)
    path, token, _ = so.verify(small.double().numpy(), None, tok[-3:].tolist(), [-1, 0, 1], [0.0] * 3, 0.7)
    assert following[1].tolist()[1] == len(path) and following[2].tolist()[1] == token
    ext.device_status()
