"""The definitions that the 8-bit cache, verification and page tests compare against (CPU)."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so


def test_e4m3_codes_are_those_of_torch():
    all_codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(all_codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(so.values(all_codes, "e4m3"), want)
    x = torch.randn(4000, dtype=torch.float64, generator=torch.Generator().manual_seed(0)) * 100
    x = torch.cat([x, x * 1e-4, torch.tensor([0.0, 448.0, -448.0, 464.0 - 17, 2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0])])
    x = x.float().clamp(-448, 448)
    want = x.to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(so.values(so.encode(x.double().numpy(), "e4m3"), "e4m3"), want)


def test_int8_codes_round_to_even_and_stay_symmetric():
    x = np.array([0.5, 1.5, -0.5, -2.5, 127.0, -127.0, 126.5, 3.49])
    assert so.values(so.encode(x, "int8"), "int8").tolist() == [0, 2, 0, -2, 127, -127, 126, 3]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("top", [0.0, 1e-30, 0.49, 0.5, 127.0, 128.0, 448.0, 449.0, 3e38, 2.0 ** -55])
def test_scales_are_the_least_powers_of_two(fmt, top):
    s = so.scale_for(top, fmt)
    assert np.log2(s) == np.floor(np.log2(s)) and top <= so.QMAX[fmt] * s
    assert s == 2.0 ** -64 or top > so.QMAX[fmt] * s / 2


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_blocks_filled_token_by_token_stay_near(fmt):
    """int8: half a step for the last rounding, less than another half for those before (each
    scale on the way is at most half the next: 1/4 + 1/8 + ...).  e4m3: a normal code is
    off by at most 2^-4 of the value once and then halves exactly; a subnormal one is rounded
    anew at every scale, by half its step, 2^-10 of the scale: 2^-10 s (1 + 1/2 + 1/4 + ...)
    < 2^-9 s.  A value may be both in turn, so the two add up."""
    rng = np.random.default_rng(1)
    codes, scales = np.zeros((1, 16, 1, 64), np.uint8), np.zeros((1, 1, 1))
    rows = rng.standard_normal((16, 1, 64)) * 2.0 ** np.arange(-3, 5, 0.5)[:, None, None]
    for n in range(1, 17):
        so.append(codes, scales, rows[n - 1:n], [0], n, 16, fmt)
    got, s = so.expand(codes, scales, fmt)[0], scales[0, 0, 0]
    assert s == so.scale_for(np.abs(rows).max(), fmt)
    bound = 1.0 * s if fmt == "int8" else 2.0 ** -4 * np.abs(rows) + s * 2.0 ** -9
    assert np.all(np.abs(got - rows) <= bound)


@pytest.mark.parametrize("kids", [1, 2, 3])
def test_verified_tokens_are_the_targets(kids):
    """Over all drafts drawn from q and all u, the first token after the root is distributed as p:
    the shares are integrals over u, taken from where the definition's tests change."""
    p, q = np.array([0.5, 0.2, 0.3, 0.0]), np.array([0.1, 0.45, 0.25, 0.2])
    share = np.zeros(4)

    def walk(weight, cover, mass, left):
        w = np.maximum(p - cover * q, 0.0)
        if left == 0:
            share[:] += weight * (w if cover else p) / (w if cover else p).sum()
            return
        refused = 0.0
        for x in range(4):
            tokens = [0] * (kids + 1)
            level = kids - left + 1
            tokens[level] = x
            ok = min(1.0, w[x] / (q[x] * mass))
            # the oracle agrees on both sides of that border
            for du, want in ((-1e-9, True), (1e-9, False)):
                if 0 <= ok + du < 1 and level == 1:
                    path, _, _ = so.verify([p] * (kids + 1), [q] * (kids + 1), tokens, [-1] + [0] * kids,
                                           [0.0] + [ok + du] + [1.0] * (kids - 1), 0.0)
                    assert (path[1:2] == [1]) == want
            share[x] += weight * q[x] * ok
            refused += weight * q[x] * (1 - ok)
        if refused > 1e-15:
            walk(refused, cover + mass, np.maximum(p - (cover + mass) * q, 0.0).sum(), left - 1)
    walk(1.0, 0.0, 1.0, kids)
    np.testing.assert_allclose(share, p, atol=1e-12)


def test_chosen_tokens_leave_the_rest():
    p = np.array([0.5, 0.3, 0.2])
    target = [p, p, p]
    assert so.verify(target, None, [0, 0, 1], [-1, 0, 0], [0, 0.49, 0.9], 0.0)[0] == [0, 1]
    assert so.verify(target, None, [0, 0, 1], [-1, 0, 0], [0, 0.5, 0.59], 0.0)[0] == [0, 2]
    path, token, w = so.verify(target, None, [0, 0, 1], [-1, 0, 0], [0, 0.5, 0.61], 0.9)
    assert path == [0] and token == 2 and w.tolist() == [0, 0, 0.2]


def test_pages_model_keeps_its_counts():
    m = so.Pages([[0, 1, -1], [0, 2, -1]], [2, 1, 1, 0, 0], [6, 5], 4, range(5))
    m.fork([0, 0])
    assert m.refs.tolist() == [2, 2, 0, 0, 0]
    assert m.reserve([9, 7]) == 0
    assert m.table.tolist() == [[0, 2, 3], [0, 1, -1]] and m.refs.tolist() == [2, 1, 1, 1, 0] and m.labels[2] == 1
    assert m.reserve([12, 13]) == 0 + 1
    m.release([0, 7])
    assert m.refs.tolist() == [1, 1, 0, 0, 0] and m.compact() == 2
