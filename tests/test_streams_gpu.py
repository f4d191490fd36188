"""Calls on a stream that is not the current one: outputs that a call allocates stay its own
until the work there has ended, whether the caller keeps them or not."""
import pytest
import torch

from cache_ops import cu, paged, same

pytestmark = pytest.mark.gpu

BUSY = 20_000_000  # cycles, about 10 ms


@pytest.fixture(scope="module")
def ext():
    from paged_kv_sink_gb300 import build
    build.build()
    import paged_kv_sink_gb300 as ext
    return ext


def case(ext, name, seed):
    """(call(stream) -> outputs that it allocates) on inputs of its own."""
    g = torch.Generator().manual_seed(seed)
    lens = [300, 77]
    k, v, table, sl = (t.cuda() for t in paged(lens, 2, 64, 16, seed=seed))
    q = torch.randn(64, 8, 64, generator=g).bfloat16().cuda()
    kn = torch.randn(64, 2, 64, generator=g).bfloat16().cuda()
    c, parents = cu([40, 24]).cuda(), torch.full((64,), -1).int().cuda()
    f, _ = ext.attn_sink_rope_freqs(64)
    pos = torch.arange(64).int().cuda()
    w = torch.rand(2, 2, 300, generator=g).cuda()
    out, lse = ext.attn_sink_fwd(q, kn, kn, None, c, c, 40, 40)
    calls = dict(
        rope=lambda s: ext.attn_sink_rope(q, kn, pos, f, stream=s),
        append=lambda s: (ext.attn_sink_rope_kv_append(q, kn, kn, k, v, table, sl, f, cu_new=c, max_new=40, stream=s),),
        tree=lambda s: ext.attn_sink_tree_paged(q, k, v, table, c, sl, parents, 40, 300, stream=s),
        weights=lambda s: ext.attn_sink_decode_paged_weights(q[:2], k, v, table, sl, w, stream=s),
        evict=lambda s: ext.attn_sink_evict_paged(k, v, table, sl, w, 64, stream=s),
        decode=lambda s: ext.attn_sink_decode_paged(q[:2], k, v, table, sl, stream=s),
        forward=lambda s: ext.attn_sink_fwd(q, kn, kn, None, c, c, 40, 40, stream=s),
        backward=lambda s: ext.attn_sink_bwd(q, kn, kn, None, out, lse, q, c, c, 40, 40, stream=s)[:3])
    state = (k, v, w)
    return calls[name], state


NAMES = ("rope", "append", "tree", "weights", "evict", "decode", "forward", "backward")


@pytest.mark.parametrize("name", NAMES)
def test_dropped_outputs_are_not_handed_on_too_early(ext, name):
    """While the stream is still busy, tensors that the caller makes behind the call get other
    memory: their contents stay, and so do the lists that an eviction's moves read."""
    call, state = case(ext, name, 1)
    before = [t.clone() for t in state]
    shapes = [(t.shape, t.dtype) for t in call(None)]
    want = [t.clone() for t in state]
    for t, b in zip(state, before):
        t.copy_(b)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    call(side)                                     # the outputs are dropped here
    mine = [torch.full(s, 5, dtype=t, device="cuda") for s, t in shapes for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.all(m == 5) for m in mine)
    for t, w in zip(state, want):
        assert same(t, w)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_dropped_while_the_current_stream_still_reads_them(ext, name):
    """The current stream goes on with the outputs; the next call on the other stream does
    not get their memory before it has read them."""
    call, _ = case(ext, name, 2)
    other, _ = case(ext, name, 3)
    want = [t.clone() for t in case(ext, name, 2)[0](None)]
    other(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    copies = [t.clone() for t in got]
    del got
    again = other(side)
    torch.cuda.synchronize()
    for a, b in zip(copies, want):
        assert torch.equal(a, b) if a.dtype == torch.int32 else same(a, b)
    del again


@pytest.mark.parametrize("name", NAMES)
def test_a_forked_stream_inside_a_capture(ext, name):
    """A call on a stream that the capture forked to, its outputs made inside the capture."""
    call, state = case(ext, name, 4)
    before = [t.clone() for t in state]
    want = [t.clone() for t in call(None)] + [t.clone() for t in state]
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = list(call(side))
        torch.cuda.current_stream().wait_stream(side)
        got = [t.clone() for t in got]
    for _ in range(2):
        for t, b in zip(state, before):
            t.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got + list(state), want):
            assert torch.equal(a, b) if a.dtype == torch.int32 else same(a, b)
