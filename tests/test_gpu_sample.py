"""sample_tokens against the oracle in 64 bits.

A token has to be the oracle's, except where u lies within 2^-40 of the kept weight of a
running sum (weights are right to 2^-50 and sums to about as much, so that neither side
is the right one there; the inputs here have next to none).  A log-probability is rounded
once to float32, which is off by at most 2^-24 of its value; its 64-bit value differs from
the oracle's by no more than a few 2^-50 of the terms it is made of, for which 2^-40 is
allowed."""
import numpy as np
import pytest
import torch

import decode_oracle as do
import prefix_scan_stream_amd as ps
from gpu_util import DEV, to_host

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def vec(values, dtype=torch.float32):
    return None if values is None else torch.tensor(np.asarray(values), dtype=dtype, device=DEV)


def check(logits, u, t, k=None, p=None, m=None, **out):
    """logits: a device matrix; the rest host vectors (float32 / int32 values)."""
    rows = logits.shape[0]
    u, t = np.asarray(u, dtype=np.float32), np.asarray(t, dtype=np.float32)
    p, m = (None if v is None else np.asarray(v, dtype=np.float32) for v in (p, m))
    tokens, lps = ps.sample_tokens(logits, vec(u), vec(t), vec(k, torch.int32), vec(p), vec(m), **out)
    tokens, lps = to_host(tokens), to_host(lps)
    x = to_host(logits.float())
    for r in range(rows):
        want, lp, margin = do.sample_row(x[r], u[r], t[r], None if k is None else k[r], None if p is None else p[r],
                                         None if m is None else m[r])
        if margin > 2.0**-40:
            where = f"row {r}: u={u[r]} t={t[r]}" + "".join(f" {n}={v[r]}" for n, v in (("k", k), ("p", p), ("m", m)) if v is not None)
            assert tokens[r] == want, where
            if np.isfinite(lp):
                assert abs(float(lps[r]) - lp) <= 2.0**-24 * abs(lp) + 2.0**-40 * (1 + abs(lp)), where
            else:
                assert lps[r] == lp, where


def rows_of(rows, vocab, dtype, seed, spread=2.0, masked=0.0, pad=0, lift=True):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, spread, (rows, vocab))
    if lift:
        hot = rng.random((rows, vocab)) < 20 / vocab
        x = np.where(hot, x + 4 + rng.exponential(3, x.shape), x)
    x[rng.random(x.shape) < masked] = -np.inf
    full = torch.zeros(rows, vocab + pad, dtype=dtype, device=DEV)
    full[:, :vocab] = torch.tensor(x, device=DEV).to(dtype)
    return full[:, :vocab]


def uniforms(rows, seed):
    u = np.random.default_rng(seed).integers(0, 1 << 24, rows) / 2.0**24
    u[:1] = 0.0
    u[1:2] = 1 - 2.0**-24
    return u


VOCABS = [1, 2, 7, 63, 64, 65, 511, 513, 1000, 8191, 8193, 50003, 131072]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", VOCABS)
def test_cuts(vocab, dtype):
    rows = 12 if vocab < 10000 else 5
    for n, (k, p, m) in enumerate([(None, None, None), (50, None, None), (None, 0.9, None), (None, None, 0.02),
                                   (40, 0.8, 0.05), (vocab // 3 + 1, 0.7, None), (vocab // 2 + 1, None, 0.001),
                                   (2000, 0.97, None)]):
        print(f"vocab={vocab} {dtype} k={k} p={p} m={m}", flush=True)
        x = rows_of(rows, vocab, DTYPES[dtype], 1000 + n + vocab, pad=(0, 1, 8, 3)[n % 4], lift=n % 2 == 0)
        r = np.random.default_rng(n)
        t = r.uniform(0.3, 1.5, rows)
        check(x, uniforms(rows, n + vocab), t, None if k is None else r.integers(max(1, k // 2), k + 1, rows),
              None if p is None else r.uniform(0.5 * p, p, rows), None if m is None else r.uniform(0, 2 * m, rows))


@pytest.mark.parametrize("dtype", DTYPES)
def test_flat_and_peaked(dtype):
    """Weights from all alike to one that leaves nothing to the others."""
    for spread in (1e-3, 0.05, 0.5, 8.0, 100.0):
        print(f"{dtype} spread={spread}", flush=True)
        x = rows_of(6, 30011, DTYPES[dtype], int(spread * 1000), spread=spread, lift=False)
        u = uniforms(6, 5)
        t = [1.0, 0.01, 0.3, 5.0, 100.0, 1.0]
        check(x, u, t)
        check(x, u, t, k=[1, 29000, 12000, 5000, 6000, 30011], p=[0.9, 0.99, 0.5, 0.3, 0.9999, 0.6])
        check(x, u, t, p=[0.05, 0.2, 0.4, 0.6, 0.8, 0.999])
        check(x, u, t, m=[1.0, 0.5, 0.1, 1e-3, 1e-6, 7.0])


@pytest.mark.parametrize("dtype", DTYPES)
def test_equal_values(dtype):
    """Cuts that fall among equal values take the lower indices: all equal, three values,
    more of them than are sorted at once and fewer; zeros of both signs are equal."""
    for vocab in (100, 5003, 40007):
        print(f"{dtype} vocab={vocab}", flush=True)
        rng = np.random.default_rng(vocab)
        x = torch.zeros(8, vocab, dtype=DTYPES[dtype], device=DEV)
        x[1] = -3.5
        x[2:5] = torch.tensor(rng.choice([0.0, 1.0, -2.0], (3, vocab)), device=DEV).to(x.dtype)
        x[5] = torch.tensor(rng.choice([0.0, -0.0], vocab), device=DEV).to(x.dtype)
        x[6] = torch.tensor(rng.choice([5.0, 5.25], vocab, p=[0.95, 0.05]), device=DEV).to(x.dtype)
        x[7, ::3] = -7.0
        u, t = uniforms(8, 3), np.full(8, 0.7)
        u[2:] = rng.random(6).astype(np.float32)
        check(x, u, t)
        check(x, u, t, k=rng.integers(1, vocab, 8))
        check(x, u, t, p=rng.uniform(0.1, 0.95, 8))
        check(x, u, t, k=rng.integers(vocab // 2, vocab, 8), p=rng.uniform(0.1, 0.95, 8), m=np.full(8, 0.2))
        check(x, u, np.zeros(8))


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked(dtype):
    """-inf, NaN and the type's lowest value; rows with one token left and with none."""
    dt = DTYPES[dtype]
    x = rows_of(12, 5003, dt, 9, masked=0.6, pad=5)
    x[0] = -torch.inf
    x[1] = torch.nan
    x[2] = -torch.inf
    x[2, 4999] = -3.0
    x[3, ::2] = torch.nan
    x[4] = torch.finfo(dt).min
    x[5, :5000] = torch.finfo(dt).min
    x[6, 1:] = torch.finfo(dt).min
    x[7] = -torch.inf
    x[7, 77] = torch.finfo(dt).min
    x[8, 100:] = -torch.inf
    x[9, 5] = torch.finfo(dt).max
    u = uniforms(12, 21)
    for t in (np.full(12, 0.9), np.zeros(12), np.full(12, 30.0)):
        check(x, u, t)
        check(x, u, t, k=np.full(12, 3))
        check(x, u, t, k=np.full(12, 5000), p=np.full(12, 0.9))
        check(x, u, t, p=np.full(12, 0.5), m=np.full(12, 0.1))
        check(x, u[::-1].copy(), t, m=np.full(12, 1e-4))


NAN_BITS = {"f32": (0x7F800001, 0x7FC00000, -0x7FFFFF, -0x400000), "f16": (0x7C01, 0x7E00, -0x3FF, -0x200),
            "bf16": (0x7F81, 0x7FC0, -0x7F, -0x40)}


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_kind_of_nan(dtype):
    """NaN of both signs, quiet and signalling, among other logits and all over a row."""
    x = rows_of(6, 9001, DTYPES[dtype], 55)
    ints = x.view(torch.int32 if dtype == "f32" else torch.int16)
    where = np.random.default_rng(5).random((6, 9001)) < 0.3
    which = np.random.default_rng(6).choice(NAN_BITS[dtype], (6, 9001))
    ints[torch.tensor(where, device=DEV)] = torch.tensor(which[where], device=DEV).to(ints.dtype)
    ints[3] = torch.tensor(which[3], device=DEV).to(ints.dtype)
    u, t = uniforms(6, 8), [1.0, 0.7, 1.3, 1.0, 0.0, 0.9]
    assert bool(x[3].isnan().all()) and int(x[0].isnan().sum()) > 1000
    check(x, u, t)
    check(x, u, t, k=np.full(6, 9))
    check(x, u, t, k=np.full(6, 4000), p=np.full(6, 0.9))
    check(x, u, t, p=np.full(6, 0.8), m=np.full(6, 0.001))
    check(x, u, t, m=np.full(6, 0.01))


def test_infinite_logits():
    """+inf logits share everything; the first of them is the greedy choice."""
    x = rows_of(4, 700, torch.float32, 4)
    x[:, [30, 31, 500]] = torch.inf
    check(x, [0.0, 0.3, 0.5, 0.9], [1.0, 1.0, 0.0, 2.0])
    check(x, [0.0, 0.3, 0.5, 0.9], [1.0, 1.0, 0.0, 2.0], k=[2, 1, 5, 699], p=[0.5, 0.9, 0.3, 0.7])


def test_values_of_the_parameters():
    """Parameters outside their usual ranges, row by row."""
    rows = 10
    x = rows_of(rows, 3001, torch.float32, 31)
    u = [-0.5, np.nan, 1.0, 2.0, 0.5, 0.5, 0.5, 0.5, 0.5, 0.25]
    t = [1.0, 1.0, 1.0, 1.0, np.nan, -1.0, np.inf, 1e-40, 1e30, 1e-6]
    check(x, u, t)
    check(x, u, t, k=[0, -1, 1, 2**31 - 1, 5, 5, 5, 5, 3001, 3002])
    check(x, u, t, p=[0.0, -1.0, np.nan, 1.0, 1.5, np.inf, 0.5, 0.5, 0.5, 0.5])
    check(x, u, t, m=[0.0, -1.0, np.nan, 1.0, 1.5, np.inf, 0.5, 0.5, 0.5, 1e-30])
    check(x, u, t, k=[0, -1, 1, 2**31 - 1, 5, 5, 5, 5, 3001, 3002], p=[0.0, -1.0, np.nan, 1.0, 1.5, np.inf, 0.5, 0.5, 0.5, 0.5],
          m=[0.0, -1.0, np.nan, 1.0, 1.5, np.inf, 0.5, 0.5, 0.5, 1e-30])


def test_long_rows():
    """Rows of more than 1024 steps (segments of several), float32 and bfloat16."""
    for dtype, vocab in ((torch.bfloat16, 1_200_007), (torch.float32, 600_011)):
        print(f"{dtype} {vocab}", flush=True)
        x = rows_of(3, vocab, dtype, 17, pad=3)
        u = [0.2, 0.7, 0.999]
        check(x, u, [1.0, 0.8, 1.3])
        check(x, u, [1.0, 0.8, 1.3], k=[600_000, 70, 5000], p=[0.9, 0.95, 0.5])
        check(x, u, [1.0, 0.8, 1.3], p=[0.3, 0.9, 0.99])


def test_many_rows():
    for rows, vocab in ((1, 131072), (13, 50003), (64, 20000), (300, 3001), (2000, 129)):
        print(f"rows={rows} vocab={vocab}", flush=True)
        x = rows_of(rows, vocab, torch.bfloat16, rows, masked=0.3)
        rng = np.random.default_rng(rows)
        u = rng.random(rows).astype(np.float32)
        t = np.where(rng.random(rows) < 0.2, 0.0, rng.uniform(0.5, 1.2, rows))
        check(x, u, t)
        check(x, u, t, k=rng.integers(1, 100, rows), p=rng.uniform(0.5, 1.0, rows), m=rng.uniform(0, 0.1, rows))


def test_one_workspace_for_calls_of_all_sizes():
    """Calls of different numbers of rows and tokens one after the other, and more rows than a launch takes."""
    for rows, vocab in ((3, 40000), (700, 600), (1, 9000), (40, 70001), (300, 1000), (20_000, 33), (5, 40000)):
        print(f"rows={rows} vocab={vocab}", flush=True)
        x = rows_of(rows, vocab, torch.float16, rows + vocab)
        rng = np.random.default_rng(rows)
        u, t = rng.random(rows).astype(np.float32), rng.uniform(0.5, 1.2, rows)
        check(x, u, t)
        check(x, u, t, k=rng.integers(1, 9, rows), p=rng.uniform(0.5, 1.0, rows))


def test_empty():
    f = torch.zeros(0, device=DEV)
    tokens, lps = ps.sample_tokens(torch.zeros(0, 10, device=DEV), f, f)
    assert tokens.shape == (0,) and lps.shape == (0,)
    f = torch.ones(3, device=DEV)
    tokens, lps = ps.sample_tokens(torch.zeros(3, 0, device=DEV), f, f)
    assert to_host(tokens).tolist() == [-1] * 3 and (to_host(lps) == -np.inf).all()


def test_one_row_for_all_and_far_rows():
    """A broadcast row; rows that start past 2^31 elements of the buffer."""
    row = rows_of(1, 4001, torch.bfloat16, 8)
    check(row.expand(7, 4001), uniforms(7, 3), np.full(7, 0.8), p=np.full(7, 0.9))
    stride = (1 << 31) + 3
    wide = torch.empty(stride + 4001, dtype=torch.bfloat16, device=DEV)
    x = wide.as_strided((2, 4001), (stride, 1))
    x.copy_(rows_of(2, 4001, torch.bfloat16, 9))
    check(x, [0.4, 0.6], [1.0, 1.0], k=[30, 3000], p=[0.9, 0.9])


def test_log_probabilities_not_wanted():
    x = rows_of(3, 500, torch.float32, 2)
    u, t = vec([0.1, 0.5, 0.9]), vec([1.0, 0.0, 1.0])
    want, _ = ps.sample_tokens(x, u, t)
    out = torch.empty(3, dtype=torch.int64, device=DEV)
    ws = torch.empty(max(256, ps.ls_sample_workspace_bytes(3, 500)), dtype=torch.uint8, device=DEV)
    ps.ls_workspace_init(ws)
    st = ps.load_library().sample_tokens(x.data_ptr(), 3, 500, 500, 0, u.data_ptr(), t.data_ptr(), None, None, None,
                                         out.data_ptr(), None, ws.data_ptr(), ws.numel(),
                                         torch.cuda.current_stream().cuda_stream)
    assert st == ps.LS_OK and torch.equal(out, want)


def test_same_bits_every_run_and_on_another_stream():
    x = rows_of(40, 30011, torch.bfloat16, 77)
    u, t = vec(uniforms(40, 7)), vec(np.full(40, 0.9))
    p, k = vec(np.linspace(0.1, 0.99, 40)), vec(np.linspace(1, 30000, 40).astype(int), torch.int32)
    first = [a.clone() for a in ps.sample_tokens(x, u, t, k, p)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for rep in range(5):
        with torch.cuda.stream(side):
            again = ps.sample_tokens(x, u, t, k, p)
        here = ps.sample_tokens(x, u, t, k, p)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, again)), rep
        assert all(torch.equal(a, b) for a, b in zip(first, here)), rep


def test_graph_replays():
    x = rows_of(9, 40009, torch.float16, 12)
    u, t = vec(uniforms(9, 1)), vec([0.0, 0.5, 0.7, 1.0, 1.2, 0.9, 0.8, 1.0, 1.0])
    k = vec([5, 50, 0, 500, 5000, 30000, 1, 40009, 64], torch.int32)
    p, m = vec(np.linspace(0.2, 1.0, 9)), vec(np.linspace(0.0, 0.05, 9))
    out, lps = torch.empty(9, dtype=torch.int64, device=DEV), torch.empty(9, device=DEV)
    want = [[a.clone() for a in ps.sample_tokens(x, u, t, *cuts)] for cuts in ((k, p, m), (), (None, p))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ps.sample_tokens(x, u, t, k, p, m, out=out, logprobs=lps)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    results = []
    with torch.cuda.graph(g):
        for cuts in ((k, p, m), (), (None, p)):
            results.append(ps.sample_tokens(x, u, t, *cuts))
    for rep in range(4):
        for a, b in results:
            a.fill_(-7)
            b.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        for got, w in zip(results, want):
            assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1]), rep
        ps.sample_tokens(x, u, t, None, p, m)
        torch.cuda.synchronize()


def test_binding_refuses():
    x = torch.zeros(4, 100, device=DEV)
    f = torch.ones(4, device=DEV)
    i = torch.ones(4, dtype=torch.int32, device=DEV)
    cases = [
        (TypeError, lambda: ps.sample_tokens(x.double(), f, f)),
        (TypeError, lambda: ps.sample_tokens(x, f.half(), f)),
        (TypeError, lambda: ps.sample_tokens(x, f, f, top_k=f)),
        (TypeError, lambda: ps.sample_tokens(x, f, f, top_p=f.double())),
        (TypeError, lambda: ps.sample_tokens(x, f, f, out=i)),
        (ValueError, lambda: ps.sample_tokens(x[0], f, f)),
        (ValueError, lambda: ps.sample_tokens(x.t(), f, f)),
        (ValueError, lambda: ps.sample_tokens(x.as_strided((4, 100), (50, 1)), f, f)),
        (ValueError, lambda: ps.sample_tokens(x, f[:3], f)),
        (ValueError, lambda: ps.sample_tokens(x, f, f[:1].expand(4))),
        (ValueError, lambda: ps.sample_tokens(x, f.cpu(), f)),
        (ps.LibscanError, lambda: ps.sample_tokens(x, f, f, logprobs=f)),
    ]
    for kind, call in cases:
        with pytest.raises(kind):
            call()
