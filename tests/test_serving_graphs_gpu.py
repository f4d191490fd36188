"""Graphs of the serving calls replayed side by side, each on the state that it was captured for."""
import pytest
import torch

from test_serving_run_gpu import NAMES, ext, one_call  # noqa: F401  (ext: the fixture)

pytestmark = pytest.mark.gpu


def as_bytes(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("names", [("many", "decode", "reserve", "few"), ("reserve", "compact", "reserve", "fork"), ("verify", "append", "release", "many")])
def test_replays_side_by_side_leave_what_the_calls_leave(ext, names):  # noqa: F811
    """Outputs, tables, counts, scales and caches after every replay are the eager call's on the same state."""
    assert set(names) <= set(NAMES)
    made = [one_call(ext, name, seed) for seed, name in enumerate(names, 7)]
    before = [[t.clone() for t in state] for _, state in made]
    want = []
    for call, state in made:
        out = [t.clone() for t in call(None)]
        want.append(out + [t.clone() for t in state])

    def restore():
        for (_, state), old in zip(made, before):
            for t, b in zip(state, old):
                as_bytes(t).copy_(as_bytes(b))
        torch.cuda.synchronize()

    graphs = []
    for call, state in made:
        restore()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = list(call(None))
        graphs.append((graph, out + list(state)))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        restore()
        for (graph, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for (_, got), w in zip(graphs, want):
            for a, b in zip(got, w):
                assert torch.equal(as_bytes(a), as_bytes(b))
    assert ext.device_status() == 0
