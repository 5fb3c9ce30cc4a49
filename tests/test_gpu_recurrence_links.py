"""gated_recurrence and its gradients where values reach far: decays near 1 or of exactly 1 and -1, over more tiles than a
group and a stretch hold, and packed rows of more channels than four chains have.  test_link_cases.py shows on the CPU
that these cases see a broken link."""
import numpy as np
import pytest
import torch

import layer_oracle as lo
import link_cases as lc
import prefix_scan_stream_amd as ps

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def host(t):
    return None if t is None else t.double().cpu().numpy()


def close(got, want, bound, what):
    err = np.abs(host(got) - want)
    allowed = lc.room(got.dtype, want, bound)
    bad = ~(err <= allowed)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst by {np.nanmax(err / allowed):.3g} of the bound"


def same(got, want, bound, what):
    """The exact value, rounded to got's type."""
    want = torch.from_numpy(np.asarray(want)).to(got.dtype)
    assert torch.equal(got.cpu(), want), f"{what}: {int((got.cpu() != want).sum())} of {want.numel()} differ"


def run(case, gating, offsets=None):
    """The five outputs, the rows behind the last sequence as they were, and the state in place."""
    x, gate, dout, state, dstate = (t.to(DEV) for t in case)
    carries = ps.recurrence_carries(x, offsets)
    out, dx, dg = (torch.full_like(x, 7.0) for _ in range(3))
    _, last = ps.gated_recurrence(x, gate, state, gating, offsets=offsets, out=out, carries=carries)
    _, _, ds = ps.gated_recurrence_backward(dout, x, gate, carries, state=state, dstate_out=dstate, gating=gating, offsets=offsets,
                                            dx=dx, dgate=dg)
    kept = state.clone()
    again, _ = ps.gated_recurrence(x, gate, kept, gating, offsets=offsets, state_out=kept, out=torch.full_like(x, 7.0))
    assert torch.equal(again, out) and torch.equal(kept, last)
    assert ps.workspace_error_flags(DEV) == 0
    return out, dx, dg, last, ds


def check_batch(case, gating, near):
    x, gate, dout, state, dstate = map(host, case)
    out, dx, dg, last, ds = run(case, gating)
    h, hb, end = lo.recurrence(x, gate, state, gating)
    (wx, wg, ws), (bx, bg, bs) = lo.gradients(x, gate, state, dout, dstate, gating)
    for got, want, bound, what in ((out, h, hb, "h"), (last, end, hb[:, -1], "state"), (dx, wx, bx, "dx"), (dg, wg, bg, "dgate"),
                                   (ds, ws, bs, "dstate")):
        near(got, want, bound, what)


def check_packed(case, gating, lengths, near, some=None):
    """Of all sequences that have tokens, or of `some`."""
    offsets = np.concatenate([[0], np.cumsum(lengths)])
    out, dx, dg, last, ds = run(case, gating, torch.from_numpy(offsets).to(DEV))
    x, gate, dout, state, dstate = case
    live = int(offsets[-1])
    for v in (out, dx, dg):
        assert bool((v[live:] == 7.0).all())
    idle = np.flatnonzero(np.asarray(lengths) == 0)
    assert torch.equal(last.cpu()[idle], state[idle]) and torch.equal(ds.cpu()[idle], dstate[idle])
    for s in np.flatnonzero(lengths) if some is None else some:
        a, z = int(offsets[s]), int(offsets[s + 1])
        xs, gs, do, st, dso = (host(t)[None] for t in (x[a:z], gate[a:z], dout[a:z], state[s], dstate[s]))
        h, hb, end = lo.recurrence(xs, gs, st, gating)
        (wx, wg, ws), (bx, bg, bs) = lo.gradients(xs, gs, st, do, dso, gating)
        for got, want, bound, what in ((out[a:z], h, hb, "h"), (last[s], end, hb[:, -1], "state"), (dx[a:z], wx, bx, "dx"),
                                       (dg[a:z], wg, bg, "dgate"), (ds[s], ws, bs, "dstate")):
            near(got, want[0], bound[0], f"{what} of sequence {s}")
    return out, dx, dg, last, ds


def batch_of(make, batch):
    cases = [make(seed) for seed in range(batch)]
    return [torch.stack(parts) for parts in list(zip(*cases))[:3]] + [torch.cat(parts) for parts in list(zip(*cases))[3:]]


# sequences of 76 tiles in front of one another, and of 22: with one or two chains a stretch is 64 tiles, with more 8
SHAPES = {2: (1, 8192 + 1500, lc.FEW), 1: (2, 2700, lc.MANY)}
LENGTHS = {2: [1, 300, 0, 5000, 63, 2900, 0, 1428], 1: [70, 0, 1500, 1, 1129]}


@pytest.mark.parametrize("dtype", lc.TYPES)
@pytest.mark.parametrize("gating", lc.GATINGS)
@pytest.mark.parametrize("levels", [1, 2])
def test_slow_decays(levels, gating, dtype):
    batch, length, widths = SHAPES[levels]
    t = lc.TYPES[dtype]
    check_batch(batch_of(lambda seed: lc.slow_case(seed, (length, widths[dtype]), gating, t), batch), gating, close)
    n = sum(LENGTHS[levels]) + 11
    check_packed(lc.slow_case(50, (n, widths[dtype]), gating, t, len(LENGTHS[levels])), gating, LENGTHS[levels], close)


@pytest.mark.parametrize("dtype", lc.TYPES)
@pytest.mark.parametrize("levels", [1, 2])
def test_exact_sums(levels, dtype):
    """Nothing is rounded before the outputs' type, so the outputs are the exact values, rounded."""
    batch, length, widths = SHAPES[levels]
    t = lc.TYPES[dtype]
    check_batch(batch_of(lambda seed: lc.exact_case(seed, (length, widths[dtype]), t), batch), "decay", same)
    n = sum(LENGTHS[levels]) + 11
    check_packed(lc.exact_case(50, (n, widths[dtype]), t, len(LENGTHS[levels])), "decay", LENGTHS[levels], same)


@pytest.mark.parametrize("dtype,channels", [("f32", 64), ("f16", 128), ("bf16", 64)])
def test_exact_sums_of_blocks_that_walk(dtype, channels):
    """More chains than 512: a block goes over its sequence, 300 tokens of it, and hands the value on itself."""
    batch, length, t = 520, 300, lc.TYPES[dtype]
    x, gate, dout, state, dstate = lc.exact_case(3, (batch * length, channels), t, batch)
    case = [v.view(batch, length, channels) for v in (x, gate, dout)] + [state, dstate]
    check_batch(case, "decay", same)


# sequences that start and end inside tiles, at their borders, and at those of groups of eight
PACKED = {
    "mixed": [0, 5, 0, 0, 130, 1, 1, 1, 300, 0, 64, 128, 2],
    "ones": [1] * 150,
    "one": [777],
    "tile ends": [16, 112, 128, 64, 64, 1, 127, 256],
    "empty": [0, 0, 0],
    "many empty": [0] * 700 + [3] + [0] * 900 + [200] + [0] * 300,
    "groups": [1024, 1, 127, 896, 128, 1, 511, 512, 1100, 0, 63, 961, 1, 0, 1],
}


@pytest.mark.parametrize("dtype", lc.TYPES)
@pytest.mark.parametrize("name", PACKED)
def test_packed_of_many_channels(dtype, name):
    """Six chains and more, with gates that forget soon, late, and both."""
    lengths, d, t = PACKED[name], lc.MANY[dtype], lc.TYPES[dtype]
    gating = lc.GATINGS[(len(name) + len(dtype)) % 3]
    behind = 37 * (len(name) % 2)
    n = sum(lengths) + behind
    r = lc.rng(len(name))
    case = list(lc.slow_case(len(name), (n, d), gating, t, len(lengths)))
    z = r.standard_normal((n, d)) * 1.5
    rate = np.exp(z - 3.0)
    soon = z + 1.0 if gating == "sigmoid" else -rate if gating == "log" else np.exp(-rate)
    case[1] = torch.where(torch.from_numpy(r.random((n, d)) < 0.3), torch.from_numpy(soon).to(t), case[1])
    check_packed(case, gating, lengths, close)


@pytest.mark.parametrize("dtype,d", [("f32", 325), ("f16", 643), ("bf16", 642)])
def test_packed_rows_that_fill_the_caches(dtype, d):
    """More rows than the caches hold are loaded by other loads: with sequences that start and end inside tiles, some of
    them against the oracle, and two halves of the call, each below that size, with the same bits."""
    t = lc.TYPES[dtype]
    half = -(-(100 << 20) // (2 * d * t.itemsize)) // 1024 * 1024 + 1024  # both: more than 192 MiB of x and gate; one: less
    assert 4 * half * d * t.itemsize >= 192 << 20 > 2 * half * d * t.itemsize
    r = lc.rng(d)
    lengths, left = [], half
    while left:
        lengths.append(min(left, int(r.choice([0, 1, 2, 63, 129, 700, 2049]))))
        left -= lengths[-1]
    n = len(lengths)
    case = list(lc.slow_case(d, (2 * half, d), "sigmoid", t, 2 * n))
    soon = r.random((2 * half, 1)) < 0.02
    case[1] = torch.where(torch.from_numpy(soon), torch.zeros((), dtype=t), case[1])
    some = [s for s in range(0, 2 * n, 7) if 0 < (lengths * 2)[s] <= 129][:12] + [lengths.index(2049), n + lengths.index(700)]
    whole = check_packed(case, "sigmoid", lengths * 2, close, some)
    for i in range(2):
        rows, seqs = slice(i * half, (i + 1) * half), slice(i * n, (i + 1) * n)
        part = [v[rows] for v in case[:3]] + [v[seqs] for v in case[3:]]
        got = run(part, "sigmoid", torch.from_numpy(np.concatenate([[0], np.cumsum(lengths)])).to(DEV))
        for a, b, of in zip(whole, got, (rows, rows, rows, seqs, seqs)):
            assert torch.equal(a[of], b)
