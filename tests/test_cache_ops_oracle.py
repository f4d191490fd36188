"""Pins of the fp64 definitions in oracle/cache_ops_oracle.py, and of the rotary
frequencies: closed forms, brute force and differences (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import attn_sink_oracle as orc
from oracle import cache_ops_oracle as co
from paged_kv_sink_gb300 import attn_sink_rope_freqs


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_depends_on_relative_positions_only(interleaved):
    g = np.random.default_rng(0)
    f, _ = attn_sink_rope_freqs(32, device="cpu")
    q, k = g.normal(size=(1, 1, 64)), g.normal(size=(1, 1, 64))
    dots = []
    for p, t in ((7, 3), (1007, 1003), (4, 0)):
        a = co.rotate(q, np.array([p]), f, interleaved)
        b = co.rotate(k, np.array([t]), f, interleaved)
        dots.append(float((a * b).sum()))
        assert np.array_equal(a[..., 32:], q[..., 32:])
    np.testing.assert_allclose(dots, dots[0], rtol=1e-10)
    # position 1 turns the first pair by one radian
    y = co.rotate(np.eye(64)[:1][None], np.array([1]), f, interleaved)
    assert y[0, 0, 0] == pytest.approx(math.cos(1)) and y[0, 0, 1 if interleaved else 16] == pytest.approx(math.sin(1))


def test_rotation_gradient_is_the_rotation_back():
    g = np.random.default_rng(1)
    f, m = attn_sink_rope_freqs(48, scaling="yarn", factor=4.0, original_len=4096, device="cpu")
    x, dy, pos = g.normal(size=(3, 2, 64)), g.normal(size=(3, 2, 64)), np.array([0, 5, 70001])
    dx = co.rotate(dy, pos, f, True, m, inverse=True)
    for idx in [(0, 0, 3), (1, 1, 20), (2, 0, 47), (2, 1, 60)]:
        e = np.zeros_like(x)
        e[idx] = 1e-6
        num = ((co.rotate(x + e, pos, f, True, m) - co.rotate(x - e, pos, f, True, m)) * dy).sum() / 2e-6
        assert num == pytest.approx(dx[idx], rel=1e-7, abs=1e-9)


def test_rope_frequencies():
    f, m = attn_sink_rope_freqs(64, device="cpu")
    assert f.dtype == torch.float64 and m == 1.0
    np.testing.assert_allclose(f.numpy(), 10000.0 ** (-np.arange(32) / 32))
    lin, _ = attn_sink_rope_freqs(64, scaling="linear", factor=4.0, device="cpu")
    np.testing.assert_allclose(lin.numpy() * 4, f.numpy())
    # "base": first pair unchanged, last divided by the factor
    b, _ = attn_sink_rope_freqs(64, scaling="base", factor=4.0, device="cpu")
    assert b[0] == f[0] and float(b[-1]) == pytest.approx(float(f[-1]) / 4)
    for kind, high in (("bands", 4.0), ("yarn", 32.0)):
        s, m = attn_sink_rope_freqs(64, scaling=kind, factor=8.0, original_len=4096, device="cpu")
        turns = 4096 * f.numpy() / (2 * math.pi)
        ratio = s.numpy() / f.numpy()
        assert np.all((ratio <= 1 + 1e-15) & (ratio >= 1 / 8 - 1e-15)) and np.all(np.diff(ratio) <= 1e-15)
        np.testing.assert_allclose(ratio[turns > high * 1.4], 1.0)
        np.testing.assert_allclose(ratio[turns < 0.7], 1 / 8)
        assert m == (1.0 if kind == "bands" else pytest.approx(0.1 * math.log(8.0) + 1))
    s, m = attn_sink_rope_freqs(64, scaling="bands", factor=8.0, original_len=4096, attn_factor=1.5, device="cpu")
    i = int(np.argmin(np.abs(turns - 2.0)))
    t = (turns[i] - 1) / 3
    assert float(s[i]) == pytest.approx(float(f[i]) * (t + (1 - t) / 8)) and m == 1.5


def test_rope_frequencies_with_an_unrounded_ramp():
    """The blend starts and ends at fractional pair indices, where a pair would make exactly 32
    and 1 turns of the original context; by default it is rounded outwards."""
    r, base, old, factor = 64, 150000.0, 4096, 32.0
    f, _ = attn_sink_rope_freqs(r, base=base, device="cpu")
    got, m = attn_sink_rope_freqs(r, base=base, scaling="yarn", factor=factor, original_len=old, round_ends=False,
                                  device="cpu")
    rounded, _ = attn_sink_rope_freqs(r, base=base, scaling="yarn", factor=factor, original_len=old, device="cpu")
    # base^(-2 i / r) old / (2 pi) = turns, solved for i
    first, last = (r / 2 * math.log(old / (2 * math.pi * n)) / math.log(base) for n in (32.0, 1.0))
    assert first != round(first) and last != round(last)
    for got_f, a, b in ((got, first, last), (rounded, math.floor(first), math.ceil(last))):
        stretched = np.clip((np.arange(32) - a) / (b - a), 0.0, 1.0)
        np.testing.assert_allclose(got_f.numpy(), f.numpy() * (1 - stretched + stretched / factor), rtol=1e-13)
    assert m == pytest.approx(0.1 * math.log(factor) + 1) and not torch.equal(got, rounded)


@pytest.mark.parametrize("kw", [dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=64, scaling="other"),
                                dict(rotary_dim=64, base=1.0), dict(rotary_dim=64, scaling="linear", factor=0.5),
                                dict(rotary_dim=2, scaling="base", factor=2.0), dict(rotary_dim=64, scaling="yarn"),
                                dict(rotary_dim=64, scaling="bands", original_len=100, low=4.0, high=4.0)])
def test_rope_frequencies_refuse(kw):
    with pytest.raises(ValueError):
        attn_sink_rope_freqs(device="cpu", **kw)


def test_tree_visibility_by_hand():
    #        0 -> 1 -> 3, 0 -> 2, and 4 on the prefix; prefix of 3 tokens
    s = co.tree_seen([-1, 0, 0, 1, -1], 3)
    want = np.array([[1, 1, 1, 1, 0, 0, 0, 0], [1, 1, 1, 1, 1, 0, 0, 0], [1, 1, 1, 1, 0, 1, 0, 0],
                     [1, 1, 1, 1, 1, 0, 1, 0], [1, 1, 1, 0, 0, 0, 0, 1]], bool)
    assert np.array_equal(s, want)
    # window: first 1 and last 2 positions.  Node 3 stands at 5 and sees 0, 4 (node 1) and itself.
    s = co.tree_seen([-1, 0, 0, 1, -1], 3, 1, 2)
    assert np.array_equal(np.nonzero(s[3])[0], [0, 4, 6]) and np.array_equal(np.nonzero(s[4])[0], [0, 2, 7])


def test_a_chain_is_causal_attention():
    g = torch.Generator().manual_seed(2)
    q = torch.randn(6, 4, 64, generator=g).bfloat16()
    k, v = (torch.randn(20, 2, 64, generator=g).bfloat16() for _ in range(2))
    sink = torch.randn(4, generator=g)
    for first, last in ((0, 0), (2, 5)):
        O, LSE, P, A = co.attend(q, k, v, co.tree_seen(list(range(-1, 5)), 14, first, last), sink, 0.125)
        ref, lse = orc.attn_fwd(q, k, v, sink, torch.tensor([0, 6]), torch.tensor([0, 20]), win_first=first,
                                win_last=last)
        np.testing.assert_allclose(O, ref, atol=1e-12)
        np.testing.assert_allclose(LSE, lse, atol=1e-12)
        np.testing.assert_allclose(P.sum(-1), 1 - np.exp(sink.numpy().astype(np.float64)[:, None] - LSE), atol=1e-12)
        assert np.all(A >= np.abs(O) - 1e-15)


def test_eviction_by_hand():
    w = [9, 1, 5, 5, 0, 5, 2, 0, 0]
    assert co.evict(w, 9, 9, 1, 2).tolist() == list(range(9))
    assert co.evict(w, 9, 5, 1, 2).tolist() == [0, 2, 3, 7, 8]      # two of the three fives: the earlier
    assert co.evict(w, 9, 3, 1, 2).tolist() == [0, 7, 8]            # nothing but the protected
    assert co.evict([np.nan, -1.0, 0.0, -0.0, np.nan], 5, 4, 0, 0).tolist() == [0, 1, 2, 3]
    assert co.evict([np.nan, -1.0, 0.0, -0.0, np.nan], 5, 2, 0, 0).tolist() == [2, 3]
