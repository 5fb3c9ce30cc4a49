"""sample_tokens where a cut by value meets long rows: few rows (their bins are made by many
blocks), flat ones (more elements in a bin than are listed at once), values that repeat, and
a bin whose elements lie in one wave's steps."""
import numpy as np
import pytest
import torch

import prefix_scan_stream_amd as ps
from gpu_util import DEV, to_host
from test_gpu_sample import DTYPES, check, rows_of, uniforms, vec

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [65535, 65536, 65537, 100003, 131072, 300007])
def test_few_rows(vocab, dtype):
    """Rows that are cut, kept whole, greedy, empty, and with min-p as well."""
    rows = 6
    x = rows_of(rows, vocab, DTYPES[dtype], vocab, pad=5)
    x[4] = -float("inf")
    u = np.random.default_rng(vocab).integers(1, 1 << 24, rows) / 2.0**24
    t, p = [0.8, 1.0, 0.0, 1.3, 1.0, 0.5], [0.9, 1.0, 0.5, 0.97, 0.9, 0.0]
    check(x, u, t, p=p)
    check(x, u, t, p=p, m=[0.0, 0.01, 0.1, 0.003, 0.2, 0.0])
    check(x, uniforms(rows, 3), t, p=[1.0, np.nan, 0.3, 1 - 2.0**-24, 2.0, 1e-30])


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_alone_and_among_many(dtype):
    """The same bits, whether few rows or many are sampled in a call."""
    x = rows_of(40, 70001, DTYPES[dtype], 8, lift=False)
    u, t = vec(uniforms(40, 8)), vec(np.linspace(0.2, 3.0, 40))
    p = vec(np.linspace(0.05, 0.999, 40))
    tokens, lps = ps.sample_tokens(x, u, t, top_p=p)
    for r in range(0, 40, 8):
        a, b = ps.sample_tokens(x[r:r + 8], u[r:r + 8], t[r:r + 8], top_p=p[r:r + 8])
        assert torch.equal(a, tokens[r:r + 8]) and torch.equal(b, lps[r:r + 8])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("spread", [0.0, 0.01, 0.3, 1.0])
def test_flat_long_rows(spread, dtype):
    vocab = 131072 if spread < 0.5 else 270001
    x = rows_of(4, vocab, DTYPES[dtype], 17, spread=spread, lift=False)
    u, t = [0.25, 0.5, 0.999, 2.0**-24], [1.0, 0.7, 1.5, 1.0]
    check(x, u, t, p=[0.9, 0.5, 0.99, 0.1])
    check(x, u, t, k=[100000, 3000, 50000, vocab])
    check(x, u, t, k=[100000, 3000, 50000, vocab], p=[0.9, 0.5, 0.99, 0.1])
    check(x, u, t, k=[60000, 7000, 900, 20000], p=[0.99999994, 0.999999, 0.9999, 1.0], m=[0.0, 0.5, 0.0, 0.9])
    check(x, np.zeros(4), t, p=[0.9, 0.5, 0.99, 0.1])


@pytest.mark.parametrize("rows", [3, 40])
def test_elements_of_one_wave(rows):
    """All of a bin's elements in every sixteenth step of 512."""
    vocab = 131072
    rng = np.random.default_rng(rows)
    x = np.full((rows, vocab), -30.0)
    at = (np.arange(vocab) // 512) % 16 == 5
    x[:, at] = rng.normal(0, 0.002, (rows, int(at.sum())))
    x[:, 7] = 4.0
    logits = torch.tensor(x, dtype=torch.float32, device=DEV)
    check(logits, uniforms(rows, 2), np.ones(rows), p=np.linspace(0.05, 0.99, rows))
    check(logits, uniforms(rows, 2), np.ones(rows), k=np.linspace(500, 8000, rows).astype(int))


def test_replays():
    """Captured calls of few rows, with eager calls of other sizes between the replays."""
    x = rows_of(5, 80000, torch.bfloat16, 4, lift=False)
    other = rows_of(100, 3000, torch.float32, 5)
    u, t, p = vec(uniforms(5, 6)), vec([0.5, 1.0, 0.0, 2.0, 1.0]), vec([0.9, 0.95, 0.9, 0.8, 1.0])
    tokens, lps = torch.empty(5, dtype=torch.int64, device=DEV), torch.empty(5, device=DEV)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        ps.sample_tokens(x, u, t, top_p=p, out=tokens, logprobs=lps)
        ps.sample_tokens(other, vec(uniforms(100, 7)), vec(np.ones(100)))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        ps.sample_tokens(x, u, t, top_p=p, out=tokens, logprobs=lps)
    for n in range(4):
        x.copy_(rows_of(5, 80000, torch.bfloat16, 40 + n, lift=False))
        u.copy_(vec(uniforms(5, 60 + n)))
        want = [to_host(v) for v in ps.sample_tokens(x, u, t, top_p=p)]
        with torch.cuda.stream(stream):
            stream.wait_stream(torch.cuda.default_stream())
            ps.sample_tokens(other, vec(uniforms(100, n)), vec(np.ones(100)), top_p=vec(np.full(100, 0.9)))
        torch.cuda.synchronize()
        tokens.fill_(-7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert (to_host(tokens) == want[0]).all() and (to_host(lps) == want[1]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [3, 40])
def test_peaked_rows(rows, dtype):
    """Most logits so far below the largest that they weigh nothing in a sum, though top-k may
    still have to count them and keep some."""
    vocab = 70000
    x = rows_of(rows, vocab, DTYPES[dtype], rows, lift=False)
    x[:, 100:110] = torch.tensor([80.0] * 9 + [79.5], device=DEV).to(x.dtype)
    x[::2, 50000] = 90.0
    x[1::3, ::5] = -float("inf")
    u, t = uniforms(rows, 9), np.full(rows, 0.6)
    for p in (0.3, 0.999999):
        check(x, u, t, p=np.full(rows, p))
        for k in (5, 1000, 60000):
            check(x, u, t, k=np.full(rows, k), p=np.full(rows, p))
    check(x, u, t, k=np.full(rows, 30000), m=np.full(rows, 1e-30))
    check(x, u, np.full(rows, 30.0), k=np.full(rows, 30000), p=np.full(rows, 0.99))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [4097, 16384, 32000, 65536, 65537, 131072])
def test_top_k_about_the_number_of_parts(vocab, dtype):
    """Around the k up to which a row's candidates come from its segments or their quarters; some rows
    with most logits masked, or with the largest ones side by side."""
    segs = -(-vocab // 512)
    ks = sorted({1, segs // 2, segs // 2 + 1, segs * 3 // 4, segs * 3 // 4 + 1, segs, segs * 3 - 1, segs * 3,
                 segs * 3 + 1, 239, 240, 241, 300} - {0})
    x = rows_of(len(ks), vocab, DTYPES[dtype], vocab + 1, lift=False)
    x[1::4, vocab // 50:] = -float("inf")
    x[2::4, 1000:1400] += 9.0
    u, t = uniforms(len(ks), 1), np.full(len(ks), 0.9)
    check(x, u, t, k=ks)
    check(x, u, t, k=ks, p=np.full(len(ks), 0.7), m=np.full(len(ks), 0.01))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [31, 500, 1025, 3001, 8192, 16384, 16385])
def test_top_k_of_short_rows(vocab, dtype):
    """The same around a short row's parts, which are finer; the parts past its end are empty."""
    segs = -(-vocab // 512)
    ks = sorted({k for n in (segs, segs * 4, segs * 16) for k in (n // 2, n // 2 + 1, n * 3 // 4, n * 3 // 4 + 1, n)} |
                {240, 241, vocab} - {0})
    ks = [k for k in ks if k > 0]
    x = rows_of(len(ks), vocab, DTYPES[dtype], vocab + 2, lift=False, pad=3)
    x[1::4, vocab // 3:] = -float("inf")
    x[2::4, :200] += 9.0
    x[3::4, vocab - 1] = float("nan")
    u, t = uniforms(len(ks), 1), np.full(len(ks), 0.9)
    check(x, u, t, k=ks)
    check(x, u, t, k=ks, p=np.full(len(ks), 0.7), m=np.full(len(ks), 0.01))
