"""Several graphs of one capture stream: each has a workspace of its own, filled by itself,
so that they may be replayed in any order, between eager calls and beside each other."""
import numpy as np
import pytest
import torch

import prefix_scan_stream_amd as ps
import workloads as wl
from gpu_util import DEV, to_dev
from test_gpu_sample import rows_of, uniforms, vec

pytestmark = pytest.mark.gpu


def work_of(size, seed):
    """Calls of every kind of workspace on inputs of about `size`; returns them as a function."""
    x = to_dev(wl.int_uniform(40 * size + 11, -1000, 1000, seed=seed))
    logits = rows_of(9, size, torch.bfloat16, seed)
    u, t = vec(uniforms(9, seed)), vec(np.linspace(0.0, 1.2, 9))
    k, p = vec(np.linspace(1, size // 2, 9).astype(int), torch.int32), vec(np.linspace(0.2, 1.0, 9))

    def work():
        kept, count = ps.compact_if(x, "lt", 0)
        return [ps.scan_exclusive(x, "sum"), ps.scan_ex(x, "sum", scheme="reduce_then_scan"), kept, count,
                ps.radix_sort(x)[0], *ps.sample_tokens(logits, u, t), *ps.sample_tokens(logits, u, t, k, p),
                *ps.sample_tokens(logits, u, t, top_p=p)]
    return work


def results(got, count_at=3):
    n = int(got[count_at])
    return [v[:n] if i == count_at - 1 else v for i, v in enumerate(got)]


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(results(got), want))


def capture(work, stream=None):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, **({} if stream is None else {"stream": stream})):
        return graph, work()


def scratch(buffers):
    """Words that no fill leaves there."""
    for ws in buffers:
        ws.fill_(0xA5)


@pytest.mark.parametrize("warm", [False, True])
def test_graphs_in_any_order(warm):
    sizes = [100_003, 70_001, 33_000]
    works = [work_of(size, 30 + i) for i, size in enumerate(sizes)]
    wants = [[v.clone() for v in results(work())] for work in works]
    stream = torch.cuda.Stream() if warm else None
    if warm:
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            works[0]()
    torch.cuda.synchronize()
    graphs, buffers = [], []
    for work in works:
        graphs.append(capture(work, stream))
        buffers.append([ws for _, ws in ps._ws_graph.values()])
    torch.cuda.synchronize()
    for ws in buffers[-1]:
        assert all(ws is not other for other in ps._ws_cache.values())
    # the later graphs' buffers come from their pools and hold anything before their first replay
    scratch(buffers[-1])
    torch.cuda.synchronize()
    for i in (2, 1, 0, 1, 2, 0):
        for v in graphs[i][1]:
            v.fill_(77)
        graphs[i][0].replay()
        torch.cuda.synchronize()
        assert same(graphs[i][1], wants[i]), i
        works[i]()
        torch.cuda.synchronize()


def test_graphs_beside_each_other():
    works = [work_of(100_003, 50), work_of(90_001, 51)]
    wants = [[v.clone() for v in results(work())] for work in works]
    graphs = [capture(work) for work in works]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for rep in range(4):
        for (graph, _), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
                graph.replay()
        works[0]()
        torch.cuda.synchronize()
        for (_, got), want in zip(graphs, wants):
            assert same(got, want), rep
            for v in got:
                v.fill_(77)
        torch.cuda.synchronize()


def test_eager_calls_on_the_capture_stream_before_the_first_replay():
    work, other = work_of(70_001, 60), work_of(60_001, 61)
    want, want_other = ([v.clone() for v in results(w())] for w in (work, other))
    stream = torch.cuda.Stream()
    graph, got = capture(work, stream)
    with torch.cuda.stream(stream):
        eager = other()
    torch.cuda.synchronize()
    assert same(eager, want_other)
    graph.replay()
    torch.cuda.synchronize()
    assert same(got, want)
