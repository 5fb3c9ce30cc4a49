"""Several host threads calling the library on one stream: the calls that are more than one
kernel (few rows of sample_tokens with top-p alone, the sort, the three-phase scans) hand
data on through the stream's workspace, and no other call's kernels may come between."""
import threading

import numpy as np
import pytest
import torch

import prefix_scan_stream_amd as ps
import workloads as wl
from gpu_util import DEV, to_dev
from test_gpu_sample import rows_of, uniforms, vec

pytestmark = pytest.mark.gpu


def sampling(rows, vocab, seed):
    x = rows_of(rows, vocab, torch.bfloat16, seed, lift=False)
    u, t, p = vec(uniforms(rows, seed)), vec(np.full(rows, 0.9)), vec(np.linspace(0.3, 0.99, rows))
    return lambda: ps.sample_tokens(x, u, t, top_p=p)


def sorting(n, seed):
    x = to_dev(wl.int_uniform(n, -10**6, 10**6, seed=seed))
    return lambda: ps.radix_sort(x)[:1]


def phases(n, seed):
    x = to_dev(wl.int_uniform(n, -1000, 1000, seed=seed))
    return lambda: [ps.scan_ex(x, "sum", scheme="scan_then_propagate")]


@pytest.mark.parametrize("kind", ["sampling", "sorting", "phases"])
def test_threads_on_one_stream(kind):
    sizes = [(1, 131072), (8, 70001), (3, 100003), (2, 65536)] if kind == "sampling" else [200_003, 90_001, 150_000, 7]
    make = {"sampling": lambda s, i: sampling(*s, i), "sorting": sorting, "phases": phases}[kind]
    calls = [make(size, 70 + i) for i, size in enumerate(sizes)]
    wants = [[v.clone() for v in call()] for call in calls]
    torch.cuda.synchronize()
    got = [[] for _ in calls]

    def work(i):
        torch.cuda.set_device(DEV)
        for _ in range(30):
            got[i].append(calls[i]())

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for i, want in enumerate(wants):
        assert len(got[i]) == 30
        assert all(torch.equal(a, b) for one in got[i] for a, b in zip(one, want)), sizes[i]
