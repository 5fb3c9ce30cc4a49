"""sample_tokens at its edges: rows that are settled before their cuts, u at and past 1, and
rows so long that the bins' rounding grows."""
import numpy as np
import pytest
import torch

import decode_oracle as do
import prefix_scan_stream_amd as ps
from gpu_util import DEV, to_host
from test_gpu_sample import DTYPES, check, rows_of, uniforms, vec

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [900, 20000, 131072])
def test_rows_that_are_settled_early(vocab, dtype):
    """Greedy rows and rows with nothing left end in one wave, the others of their block with them;
    beside rows with cuts, and the same bits each time."""
    rows = 32
    x = rows_of(rows, vocab, DTYPES[dtype], vocab + 3)
    x[1::4] = -float("inf")
    t = np.where(np.arange(rows) % 4 == 2, 0.0, 0.8)
    u = uniforms(rows, 12)
    for cuts in (dict(k=np.full(rows, 20)), dict(p=np.full(rows, 0.9)), dict(k=np.full(rows, vocab // 2), p=np.full(rows, 0.8))):
        check(x, u, t, **cuts)
        args = vec(u), vec(t), vec(cuts.get("k"), torch.int32), vec(cuts.get("p"))
        first = [to_host(v) for v in ps.sample_tokens(x, *args)]
        for _ in range(20):
            again = ps.sample_tokens(x, *args)
        assert all((a == to_host(b)).all() for a, b in zip(first, again))


def with_light_end(rows, vocab, dtype, nats, seed):
    """Logits whose last tokens, in index order, lie `nats` and a little more below the largest, and
    behind them masked ones."""
    x = rows_of(rows, vocab, dtype, seed, spread=1.0, lift=False)
    top = x.float().amax(1, keepdim=True)
    end = top - nats - torch.arange(5, device=DEV) / 4
    x[:, -8:-3] = end.to(dtype)
    x[:, -3:] = -float("inf")
    return x


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", [(5, 200), (5, 3001), (5, 20000), (5, 131072), (40, 70001), (3, 300_007)])
def test_u_of_one_and_above_takes_the_last_kept_token(rows, vocab, dtype):
    """Also where that token weighs less than the rounding of the sums, or nothing beside them."""
    u = np.resize([1.0, 1.0 + 2.0**-23, 2.0, np.inf], rows)
    for nats in (3.5, 10.0, 60.0):
        x = with_light_end(rows, vocab, DTYPES[dtype], nats, vocab)
        host = to_host(x.float())
        for t in (0.1, 1.0):
            for cuts in (dict(), dict(k=np.full(rows, vocab)), dict(k=np.full(rows, vocab - 5)), dict(k=np.full(rows, vocab // 2)),
                         dict(k=np.full(rows, 20)), dict(m=np.full(rows, 1e-35)), dict(p=np.full(rows, 0.9)),
                         dict(p=np.full(rows, 1 - 2.0**-24)), dict(k=np.full(rows, vocab - 4), m=np.full(rows, 1e-35))):
                print(f"{rows} x {vocab} {dtype} {nats} t={t} " + " ".join(cuts), flush=True)
                ks, ps_, ms = (cuts.get(n) for n in "kpm")
                tokens, lps = ps.sample_tokens(x, vec(u), vec(np.full(rows, t)), vec(ks, torch.int32), vec(ps_), vec(ms))
                tokens, lps = to_host(tokens), to_host(lps)
                for r in range(min(rows, 5)):
                    want, lp, _ = do.sample_row(host[r], u[r], np.float32(t), *(None if v is None else np.asarray(v, d)[r] for v, d in
                                                                               ((ks, np.int32), (ps_, np.float32), (ms, np.float32))))
                    assert tokens[r] == want, (r, u[r])
                    # the log-probability's one rounding, as in test_gpu_sample
                    assert abs(float(lps[r]) - lp) <= 2.0**-24 * abs(lp) + 2.0**-40 * (1 + abs(lp)), (r, u[r])


@pytest.mark.parametrize("dtype", DTYPES)
def test_u_of_one_where_a_wave_starts_with_light_tokens(dtype):
    """Without cuts: a segment whose sum is taken relative to a logit that weighs nothing, before
    the one token that does; and a row of which only the first token weighs anything."""
    vocab = 131072
    x = torch.full((4, vocab), -200.0, dtype=DTYPES[dtype], device=DEV)
    x[0, 5] = 0.0
    x[1, 70000] = 0.0
    x[2, [9, 130000]] = 0.0
    x[3, 5] = 0.0
    x[3, 130500:] = -74.0  # weighs about 2^-1068 at a temperature of 0.1
    tokens, _ = ps.sample_tokens(x, vec([1.0] * 4), vec([0.1] * 4))
    assert to_host(tokens).tolist() == [5, 70000, 130000, vocab - 1]
    # so many rows that a wave takes several segments: a sum that counts for something as a whole (2048 weights
    # of 2^-1082), where each of its weights is 0 in 64 bits
    x = torch.full((256, vocab), -200.0, dtype=DTYPES[dtype], device=DEV)
    x[:, 5] = 0.0
    x[:, -4096:-2048] = -73.5
    x[:, -2048:] = -75.0
    tokens, _ = ps.sample_tokens(x, vec([1.0] * 256), vec([0.1] * 256))
    assert to_host(tokens).tolist() == [vocab - 2049] * 256


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_equal_logits_of_a_very_long_row(dtype):
    """One logit of 0 and 2^24 equal ones of -a, whose weights all round the same way in the bins.  Kept by
    top-p are those in front of p Z, and the token is the first past u times their weight, both by division;
    p and u are such that no boundary is nearer than 16 times what the sums may be off (2^-37)."""
    vocab = (1 << 24) + 5
    n = vocab - 1
    rng = np.random.default_rng(24)
    rows = []
    while len(rows) < 4:
        a, p, u = np.float32(rng.uniform(0.5, 12)), np.float32(rng.uniform(0.1, 0.99)), np.float32(rng.uniform(0.01, 0.99))
        if dtype == "bf16":
            a = np.float32(torch.tensor(a).bfloat16().float())
        w = np.exp(-np.longdouble(a))
        z = 1 + n * w
        far = lambda at, total: abs(at - np.rint(at)) * w / total > 16 * np.longdouble(2)**-37
        cut = (np.longdouble(p) * z - 1) / w  # the equal ones in front of it are kept
        kept = int(np.ceil(cut))
        goal = (np.longdouble(u) * (1 + kept * w) - 1) / w
        if 1 < cut < n - 1 and 1 < goal and far(cut, z) and far(goal, 1 + kept * w):
            rows.append((a, p, u, 1 + int(np.floor(goal)), float(-np.longdouble(a) - np.log(1 + kept * w))))
    x = torch.empty(4, vocab, dtype=DTYPES[dtype], device=DEV)
    for r, row in enumerate(rows):
        x[r] = -float(row[0])
    x[:, 0] = 0.0
    tokens, lps = ps.sample_tokens(x, vec([row[2] for row in rows]), vec(np.ones(4)), top_p=vec([row[1] for row in rows]))
    assert to_host(tokens).tolist() == [row[3] for row in rows]
    for got, row in zip(to_host(lps), rows):
        assert abs(float(got) - row[4]) <= 2.0**-24 * abs(row[4]) + 2.0**-36
