"""Rotary positions, alone, through autograd and fused with the paged append,
against the fp64 definition.

Tolerance: the output is rounded once to bf16 (at most 2^-8 of its value); in
fp32 before it, sine and cosine (angle 2^-24, function 2^-22, factor 2^-24, all
relative to 1) and two products and a sum (2^-24 each) leave less than 2^-20 of
m (|x| + |y|) of a pair."""
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


def check(got, x, positions, f, interleaved, m=1.0, inverse=False):
    want = co.rotate(x, positions, f, interleaved, m, inverse)
    r = 2 * f.numel()
    size = np.abs(co.to_np(x))
    first = np.arange(r // 2) * 2 if interleaved else np.arange(r // 2)
    second = first + (1 if interleaved else r // 2)
    pair = np.zeros_like(size)
    pair[..., first] = pair[..., second] = size[..., first] + size[..., second]
    err = np.abs(co.to_np(got) - want)
    bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * abs(m) * pair
    bound[..., r:] = 0
    assert np.all(err <= bound), float((err - bound).max())


def rows(T, hq, hkv, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, hq, d, generator=g).bfloat16(), torch.randn(T, hkv, d, generator=g).bfloat16()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,hkv,d,r", [(1, 1, 1, 64, 64), (37, 8, 2, 64, 64), (5, 12, 12, 64, 18), (9, 3, 1, 64, 2),
                                          (300, 6, 2, 128, 128), (7, 5, 5, 128, 34), (2, 64, 8, 128, 114),
                                          (33, 40, 2, 128, 64), (3000, 4, 1, 64, 48), (9, 700, 301, 64, 64)])
def test_rope_matches_definition(ext, T, hq, hkv, d, r, interleaved):
    q, k = rows(T, hq, hkv, d)
    g = torch.Generator().manual_seed(1)
    pos = torch.randint(-5, 1 << 20, (T,), generator=g).int()
    f, m = ext.attn_sink_rope_freqs(r, scaling="yarn", factor=8.0, original_len=4096)
    for inverse in (False, True):
        yq, yk = ext.attn_sink_rope(q.cuda(), k.cuda(), pos.cuda(), f, interleaved, m, inverse)
        check(yq, q, pos, f, interleaved, m, inverse)
        check(yk, k, pos, f, interleaved, m, inverse)
    only, none = ext.attn_sink_rope(q.cuda(), None, pos.cuda(), f, interleaved, m)
    check(only, q, pos, f, interleaved, m)
    assert none is None


def test_rope_at_the_ends_of_int32(ext):
    q, k = rows(4, 2, 2, 64)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 1 << 30], dtype=torch.int32)
    f, _ = ext.attn_sink_rope_freqs(64)
    yq, _ = ext.attn_sink_rope(q.cuda(), k.cuda(), pos.cuda(), f)
    # the frequency itself is a double: 2^31 positions amplify its last bit (2^-53) to 2^-22 rad, and numpy's
    # reduction of the angle (2^-53 of 2^31) by as much: compare at 2^-20 on top of check()'s bound
    want = co.rotate(q, pos, f)
    err = np.abs(co.to_np(yq) - want)
    assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * 10)
    check(yq[2:3], q[2:3], pos[2:3], f, False)
    assert same(yq[2].cpu(), q[2])  # position 0: no turn


def test_rope_angles_keep_their_documented_accuracy(ext):
    """An angle is off by at most 1e-7 + |p| f 2^-52 rad.  A head of ones and zeros turns into its
    cosines and sines; at positions where one of them nearly vanishes the bf16 output shows
    the angle's error itself.  Beside it: bf16 rounding (2^-8 of the value) and sincospif (2 ulp,
    2^-22 of the value).  The exact angles are reduced with 50 digits."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    turn = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582")
    f, _ = ext.attn_sink_rope_freqs(64)
    near = []   # positions whose first pairs come closest to a multiple of a quarter turn
    p = np.concatenate([np.arange(1, 300000), 2 ** 31 - 1 - np.arange(300000)])
    for fi in f.cpu().tolist()[:4]:
        quarters = p.astype(np.longdouble) * np.longdouble(fi) / np.longdouble(np.pi / 2)
        near += p[np.argsort(np.abs(quarters - np.rint(quarters)))[:20]].tolist()
    pos = near + [-x for x in near] + [0, 1, -1, 2 ** 31 - 1, -2 ** 31]
    x = torch.zeros(len(pos), 1, 64).bfloat16()
    x[..., :32] = 1.0
    y, _ = ext.attn_sink_rope(x.cuda(), None, torch.tensor(pos).int().cuda(), f)
    y = co.to_np(y)[:, 0]
    for row, t in enumerate(pos):
        for i, fi in enumerate(f.cpu().tolist()):
            a = float((Decimal(t) * Decimal(fi)).remainder_near(turn))
            slack = 1e-7 + abs(t) * fi * 2.0 ** -52
            for got, want in ((y[row, i], np.cos(a)), (y[row, 32 + i], np.sin(a))):
                assert abs(got - want) <= (2.0 ** -8 + 2.0 ** -22) * (abs(want) + slack) + slack, (t, i)


@pytest.mark.parametrize("interleaved,r", [(False, 64), (True, 64), (False, 22), (True, 22)])
def test_rope_in_place_on_a_packed_buffer(ext, interleaved, r):
    """Column ranges of a packed (T, hq + 2 hkv, d) buffer, rotated in place, equal the
    contiguous call bit for bit; values and the dimensions past r keep their bits."""
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(50, 8 + 4, 64, generator=g).bfloat16()
    qkv[3, 5, 40] = float("inf")
    qkv[4, 9, 63] = float("nan")
    pos = torch.arange(50).int()
    f, _ = ext.attn_sink_rope_freqs(r)
    dev = qkv.cuda()
    want_q, want_k = ext.attn_sink_rope(dev[:, :8].contiguous(), dev[:, 8:10].contiguous(), pos.cuda(), f, interleaved)
    ext.attn_sink_rope(dev[:, :8], dev[:, 8:10], pos.cuda(), f, interleaved, q_out=dev[:, :8], k_out=dev[:, 8:10])
    got = dev.cpu()
    assert same(got[:, :8], want_q.cpu()) and same(got[:, 8:10], want_k.cpu()) and same(got[:, 10:], qkv[:, 10:])
    if r < 64:
        assert same(got[:, :10, r:], qkv[:, :10, r:])


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_gradient(ext, interleaved):
    q, k = rows(40, 4, 2, 64, seed=4)
    dq, dk = rows(40, 4, 2, 64, seed=5)
    pos = torch.arange(100, 140).int()
    f, m = ext.attn_sink_rope_freqs(48, scaling="yarn", factor=4.0, original_len=64)
    ql, kl = q.cuda().requires_grad_(), k.cuda().requires_grad_()
    yq, yk = ext.attn_sink_rope_func(ql, kl, pos.cuda(), f, interleaved, m)
    check(yq.detach(), q, pos, f, interleaved, m)
    gq, gk = torch.autograd.grad((yq, yk), (ql, kl), (dq.cuda(), dk.cuda()))
    check(gq, dq, pos, f, interleaved, m, inverse=True)
    check(gk, dk, pos, f, interleaved, m, inverse=True)
    # against differences of the fp64 definition, on a few entries
    for idx in [(0, 0, 3), (7, 3, 30), (39, 2, 50)]:
        e = np.zeros(q.shape)
        e[idx] = 1e-6
        x = co.to_np(q)
        num = ((co.rotate(x + e, pos, f, interleaved, m) - co.rotate(x - e, pos, f, interleaved, m)) * co.to_np(dq)).sum() / 2e-6
        assert abs(float(gq[idx]) - num) <= 2.0 ** -8 * abs(num) + 2.0 ** -19 * 10
    # only one of the two needs a gradient, or receives one; no keys; a shared (expanded) query row
    (gk2,) = torch.autograd.grad(ext.attn_sink_rope_func(q.cuda(), kl, pos.cuda(), f, interleaved, m)[1], (kl,), (dk.cuda(),))
    assert same(gk2, gk)
    (gq2,) = torch.autograd.grad(ext.attn_sink_rope_func(ql, kl, pos.cuda(), f, interleaved, m)[0], (ql,), (dq.cuda(),))
    assert same(gq2, gq)
    (gq3,) = torch.autograd.grad(ext.attn_sink_rope_func(ql, None, pos.cuda(), f, interleaved, m), (ql,), (dq.cuda(),))
    assert same(gq3, gq)
    one = q[:1].cuda().requires_grad_()
    y = ext.attn_sink_rope_func(one.expand(40, 4, 64).contiguous(), None, pos.cuda(), f, interleaved, m)
    (g1,) = torch.autograd.grad(y, (one,), (dq.cuda(),))
    # 40 bf16 gradients summed by torch: one rounding each and one of the sum
    want = co.rotate(dq, pos, f, interleaved, m, inverse=True)
    assert np.all(np.abs(co.to_np(g1) - want.sum(0, keepdims=True)) <= 2.0 ** -7 * np.abs(want).sum(0, keepdims=True))


@pytest.mark.parametrize("ahead", [1, 8])
def test_rope_gradient_from_a_flat_buffer(ext, ahead):
    # the gradient is a piece of a flat buffer, aligned to 2 bytes or to 16
    q, _ = rows(9, 3, 1, 64, seed=6)
    dq, _ = rows(9, 3, 1, 64, seed=7)
    pos = torch.arange(9).int()
    f, _ = ext.attn_sink_rope_freqs(64)
    ql = q.cuda().requires_grad_()
    y = ext.attn_sink_rope_func(ql, None, pos.cuda(), f)
    other = torch.zeros(ahead, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    flat = torch.cat([other, y.reshape(-1)])
    flat.backward(torch.cat([torch.zeros(ahead).bfloat16(), dq.reshape(-1)]).cuda())
    check(ql.grad, dq, pos, f, False, inverse=True)


def test_rope_gradient_of_the_gradient(ext):
    q, k = rows(6, 2, 1, 64, seed=6)
    pos, (f, _) = torch.arange(6).int().cuda(), ext.attn_sink_rope_freqs(64)
    ql, w = q.cuda().requires_grad_(), q.cuda().requires_grad_()
    y = ext.attn_sink_rope_func(ql, None, pos, f)
    (g,) = torch.autograd.grad(y, (ql,), (w,), create_graph=True)
    (gw,) = torch.autograd.grad(g, (w,), (k.expand(6, 2, 64).contiguous().cuda(),))
    check(gw, k.expand(6, 2, 64), pos.cpu(), f, False)


@pytest.mark.parametrize("interleaved,r,d,page", [(False, 64, 64, 16), (True, 32, 64, 7), (False, 128, 128, 64),
                                                  (False, 34, 128, 8), (True, 114, 128, 16)])
@pytest.mark.parametrize("new", [[5, 0, 130, 1, 17], [1, 1, 1, 1, 1]])
def test_rope_append_equals_rope_then_append(ext, interleaved, r, d, page, new):
    old = [0, 40, 9, 16, 3]
    hq, hkv = 6, 2
    lens = [a + b for a, b in zip(old, new)]
    k_cache, v_cache, table, sl = paged(lens, hkv, d, page, seed=7)
    T = sum(new)
    q, k = rows(T + 3, hq, hkv, d, seed=8)     # three rows of padding behind the last request
    v = rows(T + 3, hq, hkv, d, seed=9)[1]
    c = cu(new)
    pos = torch.cat([torch.arange(a, a + b) for a, b in zip(old, new)] + [torch.zeros(3, dtype=torch.int64)]).int()
    f, m = ext.attn_sink_rope_freqs(r, scaling="bands", factor=8.0, original_len=4096, attn_factor=1.25)
    kc, vc, kw, vw = (x.clone().cuda() for x in (k_cache, v_cache, k_cache, v_cache))
    q_out = torch.full_like(q, 7.0).cuda()
    ext.attn_sink_rope_kv_append(q.cuda(), k.cuda(), v.cuda(), kc, vc, table.cuda(), sl.cuda(), f, cu_new=c.cuda(),
                                 max_new=max(new), interleaved=interleaved, attn_scale=m, q_out=q_out)
    yq, yk = ext.attn_sink_rope(q.cuda(), k.cuda(), pos.cuda(), f, interleaved, m)
    check(yk, k, pos, f, interleaved, m)
    ext.attn_sink_kv_append(yk[:T].contiguous(), v[:T].contiguous().cuda(), kw, vw, table.cuda(), sl.cuda(), c.cuda(),
                            max(new))
    assert same(kc, kw) and same(vc, vw)       # every other slot (NaN) is untouched too
    assert same(q_out[:T], yq[:T]) and torch.all(q_out[T:] == 7.0)
    # given positions (a drafted tree's), and one row a request without cu_new
    pos2 = pos.flip(0).contiguous()
    ext.attn_sink_rope_kv_append(q.cuda(), k.cuda(), v.cuda(), kc, vc, table.cuda(), sl.cuda(), f, cu_new=c.cuda(),
                                 interleaved=interleaved, attn_scale=m, positions=pos2.cuda(), q_out=q_out)
    yq, yk = ext.attn_sink_rope(q.cuda(), k.cuda(), pos2.cuda(), f, interleaved, m)
    ext.attn_sink_kv_append(yk[:T].contiguous(), v[:T].contiguous().cuda(), kw, vw, table.cuda(), sl.cuda(), c.cuda(),
                            max(new))
    assert same(kc, kw) and same(vc, vw) and same(q_out[:T], yq[:T])
    if max(new) == 1:
        q1, k1, v1 = (x[:T].contiguous().cuda() for x in (q, k, v))
        y1 = ext.attn_sink_rope_kv_append(q1, k1, v1, kc, vc, table.cuda(), sl.cuda(), f, interleaved=interleaved,
                                          attn_scale=m)
        check(y1, q[:T], pos[:T], f, interleaved, m)
    assert ext.device_status() == 0


def test_rope_append_skips_bad_rows(ext):
    """Bad page ids, more new rows than tokens and rows past max_new or the tensors'
    end: skipped, with a status bit; the other rows are written."""
    k_cache, v_cache, table, sl = paged([20, 20, 20], 2, 64, 16, seed=10)
    q, k = rows(9, 2, 2, 64, seed=11)
    f, _ = ext.attn_sink_rope_freqs(64)
    ext.device_status()

    def call(table, sl, new, max_new, total=None):
        kc, vc = k_cache.clone().cuda(), v_cache.clone().cuda()
        t = slice(0, total)
        ext.attn_sink_rope_kv_append(q[t].cuda(), k[t].cuda(), k[t].cuda(), kc, vc, table.cuda(), sl.cuda(), f,
                                     cu_new=cu(new).cuda(), max_new=max_new)
        return kc.cpu(), ext.device_status()

    good, status = call(table, sl, [3, 3, 3], 3)
    assert status == 0
    bad = table.clone()
    bad[1, 1] = 1000
    kc, status = call(bad, sl, [3, 3, 3], 3)
    assert status == ext._lib.DEV_PAGE_OOB
    for b in (0, 2):
        assert same(kc[table[b, :2].long()], good[table[b, :2].long()])
    assert same(kc[table[1, :2].long()], k_cache[table[1, :2].long()])
    kc, status = call(table, torch.tensor([20, 2, 20], dtype=torch.int32), [3, 3, 3], 3)
    assert status == ext._lib.DEV_SEQLEN_OOB
    assert same(kc[table[0, :2].long()], good[table[0, :2].long()])
    kc, status = call(table, sl, [3, 9, -3], 3)   # request 1 has 9 rows, the grid covers 8 at most
    assert status & ext._lib.DEV_SEQLEN_OOB
    kc, status = call(table, sl, [3, 3, 3], 3, total=7)  # cu_new says 9 rows, the tensors hold 7
    assert status == ext._lib.DEV_SEQLEN_OOB


def test_rope_training_step_in_a_graph(ext):
    """Forward and gradient captured together, replayed on new gradients."""
    q, k = (x.cuda().requires_grad_() for x in rows(50, 4, 2, 64, seed=14))
    dq, dk = (x.cuda() for x in rows(50, 4, 2, 64, seed=15))
    pos, (f, m) = torch.arange(50).int().cuda(), ext.attn_sink_rope_freqs(64)
    torch.autograd.grad(ext.attn_sink_rope_func(q, k, pos, f), (q, k), (dq, dk))  # no eager graph stays alive
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = ext.attn_sink_rope_func(q, k, pos, f)
        got = torch.autograd.grad(y, (q, k), (dq, dk))
    dq.mul_(2.0)
    g.replay()
    torch.cuda.synchronize()
    want = ext.attn_sink_rope(dq, dk, pos, f, inverse=True)
    assert same(got[0], want[0]) and same(got[1], want[1])
    want = ext.attn_sink_rope(q.detach(), k.detach(), pos, f)
    assert same(y[0].detach(), want[0]) and same(y[1].detach(), want[1])


def test_rope_in_a_graph_and_on_another_stream(ext):
    q, k = rows(64, 8, 2, 64, seed=12)
    f, _ = ext.attn_sink_rope_freqs(64)
    q, k, pos = q.cuda(), k.cuda(), torch.arange(64).int().cuda()
    want = ext.attn_sink_rope(q, k, pos, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ext.attn_sink_rope(q, k, pos, f, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert same(got[0], want[0]) and same(got[1], want[1])
    out = [torch.empty_like(q), torch.empty_like(k)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ext.attn_sink_rope(q, k, pos, f, q_out=out[0], k_out=out[1])
    pos += 5
    g.replay()
    want = ext.attn_sink_rope(q, k, pos, f)
    assert same(out[0], want[0]) and same(out[1], want[1])


@pytest.mark.parametrize("most", [3, 3001])
def test_rope_append_leaves_rows_past_max_new(ext, most):
    """A request with one row more than max_new: that row is left out, in the caches and in
    q_out, and the status says so, however many rows the batch has in all (a block takes 1
    row of a small batch, 8 of a large one)."""
    new = [most + 1, most, most, most]
    k_cache, v_cache, table, sl = paged(new, 2, 64, 16, seed=16)
    q, k = rows(sum(new), 4, 2, 64, seed=17)
    f, _ = ext.attn_sink_rope_freqs(64)
    ext.device_status()
    got = []
    for bound in (most, most + 1):
        kc, vc, q_out = k_cache.clone().cuda(), v_cache.clone().cuda(), torch.full_like(q, 7.0).cuda()
        ext.attn_sink_rope_kv_append(q.cuda(), k.cuda(), k.cuda(), kc, vc, table.cuda(), sl.cuda(), f,
                                     cu_new=cu(new).cuda(), max_new=bound, q_out=q_out)
        got.append((kc.cpu().view(-1, 2, 64), vc.cpu().view(-1, 2, 64), q_out.cpu(), ext.device_status()))
    (kc, vc, q_out, status), (want_k, want_v, want_q, fine) = got
    assert fine == 0 and status == ext._lib.DEV_SEQLEN_OOB
    last = int(co.slot(table[0].numpy(), 16, most))
    for g, want, before, at in ((kc, want_k, k_cache.view(-1, 2, 64), last), (vc, want_v, v_cache.view(-1, 2, 64), last),
                                (q_out, want_q, torch.full_like(q, 7.0), most)):
        assert same(g[at], before[at])
        assert same(torch.cat([g[:at], g[at + 1:]]), torch.cat([want[:at], want[at + 1:]]))
