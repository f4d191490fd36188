"""The status words of all units, read in one call."""
import time

import pytest
import torch

from cache_ops import cu, paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ext():
    from paged_kv_sink_gb300 import build
    build.build()
    import paged_kv_sink_gb300 as ext
    return ext


def raisers(ext):
    """Calls that raise a bit each, in units of their own."""
    D = ext._lib
    k, v, table, sl = (t.cuda() for t in paged([40, 20], 2, 64, 16))
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    bad = torch.full_like(table, 99)
    refs = torch.ones(k.shape[0], dtype=torch.int32, device="cuda")
    p = torch.rand(2, 50, device="cuda")
    u = torch.rand(2, device="cuda")
    k8, v8 = (torch.zeros(k.shape, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones(k.shape[0], 1, 2, device="cuda") for _ in range(2))
    rows = torch.full((2, 2, 64), float("inf"), dtype=torch.bfloat16, device="cuda")
    return [(D.DEV_PAGE_OOB, lambda: ext.attn_sink_decode_paged(q, k, v, bad, sl)),
            (D.DEV_TREE, lambda: ext.attn_sink_tree_paged(q, k, v, table, cu([2, 0]).cuda(), i32([40, 20]), i32([-1, 7]), 2, 40)),
            (D.DEV_VALUE, lambda: ext.attn_sink_kv_append_q8(rows, rows, k8, v8, ks, vs, table, sl)),
            (D.DEV_PROB, lambda: ext.attn_sink_verify_draft(p, i32([0, 50]), None, cu([2]).cuda(), u, u[:1], 2)),
            (D.DEV_POOL, lambda: ext.attn_sink_pages_release(table.clone(), refs, sl, sl + 1, 16))]


def test_bits_of_several_units_come_together_and_once(ext):
    calls = raisers(ext)
    ext.device_status()
    for n in range(1, 1 << len(calls)):
        want = 0
        for i, (bit, call) in enumerate(calls):
            if n >> i & 1:
                want |= bit
                call()
        assert ext.device_status() == want
        assert ext.device_status() == 0


def test_the_status_waits_for_its_stream(ext):
    calls, side = raisers(ext), torch.cuda.Stream()
    ext.device_status()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        calls[4][1]()
        assert ext.device_status() == calls[4][0]
    assert ext.device_status() == 0


def test_a_status_costs_no_more_than_a_few_reads(ext):
    """However many units there are: one launch, one copy, one wait."""
    x = torch.zeros(1, dtype=torch.int32, device="cuda")

    def fastest(call):
        best = float("inf")
        for _ in range(200):
            torch.cuda.synchronize()
            t = time.perf_counter()
            call()
            best = min(best, time.perf_counter() - t)
        return best

    assert fastest(ext.device_status) <= 5 * fastest(lambda: x.add_(1).item())
