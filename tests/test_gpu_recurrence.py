"""gated_recurrence and its gradients on the GPU against the token-by-token oracle in 64 bits."""
import numpy as np
import pytest
import torch

import layer_oracle as lo
import prefix_scan_stream_amd as ps

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
GATINGS = ["decay", "log", "sigmoid"]


def rng(seed):
    return np.random.default_rng(20260925 + seed)


def make(r, shape, dtype):
    return torch.from_numpy(r.standard_normal(shape)).to(dtype)


def gates(r, shape, gating, dtype):
    z = r.standard_normal(shape) * 1.5
    rate = np.exp(z - 3.0)
    v = z + 1.0 if gating == "sigmoid" else -rate if gating == "log" else np.exp(-rate) * np.sign(r.random(shape) - 0.1)
    return torch.from_numpy(v).to(dtype)


def host(t):
    return None if t is None else t.double().cpu().numpy()


def dev(t):
    return None if t is None else t.to(DEV)


def close(got, want, bound, what):
    """Within `bound` before the rounding to got's type, and half a step of that."""
    eps = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    tiny = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps
    err = np.abs(host(got) - want)
    # results near float32's smallest normal value are flushed or lose bits
    room = bound * (1 + eps) + np.abs(want) * eps + tiny + 1e-37
    bad = ~(err <= room)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off, worst by {np.nanmax(err / room):.3g} of the bound"


def check(x, gate, state, gating, dout=None, dstate_out=None, place=lambda t: t.to(DEV), outs=None):
    """Forward and backward of sequences x tokens x channels (host tensors)."""
    h, hb, last = lo.recurrence(host(x), host(gate), host(state), gating)
    gx, gg, gs = place(x), place(gate), dev(state)
    carries = ps.recurrence_carries(gx)
    kw = {} if outs is None else dict(out=outs[0])
    out, state_out = ps.gated_recurrence(gx, gg, state=gs, gating=gating, carries=carries, **kw)
    close(out, h, hb, "h")
    final_bound = hb[:, -1] if x.shape[1] else 0 * last
    close(state_out, last, final_bound, "state")
    plain, _ = ps.gated_recurrence(gx, gg, state=gs, gating=gating)
    assert torch.equal(plain, out)  # keeping carries changes nothing
    if dout is None:
        return
    want, bound = lo.gradients(host(x), host(gate), host(state), host(dout), host(dstate_out), gating)
    kw = {} if outs is None else dict(dx=outs[1], dgate=outs[2])
    got = ps.gated_recurrence_backward(place(dout), gx, gg, carries, state=gs, dstate_out=dev(dstate_out), gating=gating, **kw)
    for g, w, b, name in zip(got, want, bound, ("dx", "dgate", "dstate")):
        close(g, w, b, name)
    assert ps.workspace_error_flags(DEV) == 0


LENGTHS = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 257, 1000, 2050]
CHANNELS = [1, 2, 3, 63, 64, 65, 128, 130, 257]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("length", LENGTHS)
def test_lengths(dtype, length):
    i = LENGTHS.index(length)
    for k, gating in enumerate(GATINGS):
        r = rng(100 * i + k)
        batch, channels = 1 + i % 3, CHANNELS[(i + 3 * k) % len(CHANNELS)]
        shape, t = (batch, length, channels), TYPES[dtype]
        some = (i + k) % 2 == 0
        state = make(r, (batch, channels), torch.float32) if some else None
        dstate = make(r, (batch, channels), torch.float32) if (i + k) % 3 == 0 else None
        check(make(r, shape, t), gates(r, shape, gating, t), state, gating, make(r, shape, t), dstate)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("channels", CHANNELS + [1000, 4096])
def test_channels(dtype, channels):
    for k, gating in enumerate(GATINGS):
        r = rng(5000 + channels + k)
        shape, t = (2, 150 + k, channels), TYPES[dtype]
        check(make(r, shape, t), gates(r, shape, gating, t), make(r, (2, channels), torch.float32), gating, make(r, shape, t),
              make(r, (2, channels), torch.float32))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("gating", GATINGS)
def test_a_token_each(dtype, gating):
    for batch, channels, wide in ((1, 2048, 0), (300, 64, 0), (7, 1001, 0), (5, 96, 1), (3, 8, 8)):
        r = rng(batch + channels)
        t = TYPES[dtype]
        x, g = make(r, (batch, channels), t), gates(r, (batch, channels), gating, t)
        state = make(r, (batch, channels), torch.float32)
        h, hb, last = lo.recurrence(host(x)[:, None], host(g)[:, None], host(state), gating)
        both = torch.empty(batch, 2 * channels + wide, dtype=t, device=DEV)
        gx, gg = both[:, :channels], both[:, channels + wide:]
        gx.copy_(x), gg.copy_(g)
        out, state_out = ps.gated_recurrence(gx, gg, state=dev(state), gating=gating)
        close(out, h[:, 0], hb[:, 0], "h")
        close(state_out, last, hb[:, 0], "state")
        # the same as sequences of one token, and with the state in place
        kept = dev(state)
        three, _ = ps.gated_recurrence(gx[:, None], gg[:, None], state=kept, gating=gating, state_out=kept)
        assert torch.equal(three[:, 0], out) and torch.equal(kept, state_out)
        carries = ps.recurrence_carries(gx)
        ps.gated_recurrence(gx, gg, state=dev(state), gating=gating, carries=carries)
        assert torch.equal(carries.cpu(), state)


PACKED = {
    "mixed": [0, 5, 0, 0, 130, 1, 1, 1, 300, 0, 64, 128, 2],
    "ones": [1] * 150,
    "one": [777],
    "tile ends": [16, 112, 128, 64, 64, 1, 127, 256],
    "empty": [0, 0, 0],
    "one token": [0, 1, 0],
    "many empty": [0] * 700 + [3] + [0] * 900 + [200] + [0] * 300,
    "long": [3000, 1, 500],
    # at the borders of tiles, groups of tiles and stretches of groups, and inside them
    "stretches": [8192, 1, 127, 896, 128, 7168, 1, 4095, 4096, 9000, 0, 63],
}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", PACKED)
@pytest.mark.parametrize("behind", [0, 37])
def test_packed(dtype, name, behind):
    lengths, t = PACKED[name], TYPES[dtype]
    gating = GATINGS[(len(name) + behind) % 3]
    r = rng(len(name) * 7 + behind)
    offsets = np.concatenate([[0], np.cumsum(lengths)])
    n, s, d = int(offsets[-1]) + behind, len(lengths), 70
    x, g, dout = make(r, (n, d), t), gates(r, (n, d), gating, t), make(r, (n, d), t)
    state, dstate_out = make(r, (s, d), torch.float32), make(r, (s, d), torch.float32)
    off = torch.from_numpy(offsets).to(DEV)
    gx, gg = dev(x), dev(g)
    for st, dso in ((state, dstate_out), (None, None)):
        out = torch.full((n, d), 7.0, dtype=t, device=DEV)
        dx, dg = out.clone(), out.clone()
        carries = ps.recurrence_carries(gx, off)
        gs = dev(st)
        _, state_out = ps.gated_recurrence(gx, gg, state=gs, gating=gating, offsets=off, out=out, carries=carries)
        _, _, dstate = ps.gated_recurrence_backward(dev(dout), gx, gg, carries, state=gs, dstate_out=dev(dso), gating=gating,
                                                    offsets=off, dx=dx, dgate=dg)
        live = int(offsets[-1])
        for v in (out, dx, dg):
            assert bool((v[live:] == 7.0).all())
        idle = np.flatnonzero(np.array(lengths) == 0)
        zero = torch.zeros(s, d)
        assert torch.equal(state_out.cpu()[idle], (zero if st is None else st)[idle])
        assert torch.equal(dstate.cpu()[idle], (zero if dso is None else dso)[idle])
        fwd = lo.packed(lambda a, b, c: lo.recurrence(a, b, c, gating), offsets, (host(x), True), (host(g), True), (host(st), False))
        for q, a, b, (h, hb, last) in fwd:
            close(out[a:b], h[0], hb[0], f"h of sequence {q}")
            close(state_out[q], last[0], hb[0, -1], f"state of sequence {q}")
        bwd = lo.packed(lambda a, b, c, e, f: lo.gradients(a, b, c, e, f, gating), offsets, (host(x), True), (host(g), True),
                        (host(st), False), (host(dout), True), (host(dso), False))
        for q, a, b, ((wx, wg, ws), (bx, bg, bs)) in bwd:
            close(dx[a:b], wx[0], bx[0], f"dx of sequence {q}")
            close(dg[a:b], wg[0], bg[0], f"dgate of sequence {q}")
            close(dstate[q], ws[0], bs[0], f"dstate of sequence {q}")
        if st is not None:  # in place
            again = torch.full((n, d), 7.0, dtype=t, device=DEV)
            kept = dev(st)
            ps.gated_recurrence(gx, gg, state=kept, gating=gating, offsets=off, out=again, state_out=kept)
            assert torch.equal(kept, state_out) and torch.equal(again, out)
    assert ps.workspace_error_flags(DEV) == 0


@pytest.mark.parametrize("dtype", TYPES)
def test_strides(dtype):
    """Halves of one projection, time-major layout, a slice of a longer batch, rows at odd elements,
    outputs in columns of one matrix, one gate for all sequences."""
    t, shape = TYPES[dtype], (3, 140, 66)
    for k, gating in enumerate(GATINGS):
        r = rng(900 + k)
        x, g, dout = make(r, shape, t), gates(r, shape, gating, t), make(r, shape, t)
        state = make(r, (3, 66), torch.float32)

        def fused(v):
            big = torch.zeros(*shape[:2], 3 * 66, dtype=t, device=DEV)
            big[..., 66:132] = v.to(DEV)
            return big[..., 66:132]

        def time_major(v):
            return v.to(DEV).transpose(0, 1).contiguous().transpose(0, 1)

        def cut(v):
            big = torch.zeros(5, 200, 70, dtype=t, device=DEV)
            big[1:4, 20:160, 3:69] = v.to(DEV)
            return big[1:4, 20:160, 3:69]

        for place in (fused, time_major, cut):
            both = torch.zeros(*shape[:2], 3 * 66, dtype=t, device=DEV)
            outs = (time_major(torch.zeros(shape, dtype=t)), both[..., :66], both[..., 132:])
            check(x, g, state, gating, dout, state, place, outs)
            assert bool((both[..., 66:132] == 0).all())
        one = g[:1].to(DEV).expand(shape)
        out, _ = ps.gated_recurrence(x.to(DEV), one, gating=gating)
        h, hb, _ = lo.recurrence(host(x), host(g[:1]).repeat(3, 0), None, gating)
        close(out, h, hb, "one gate for all")


def test_no_tokens_and_no_sequences():
    for gating in GATINGS:
        state = torch.randn(4, 33, device=DEV)
        x = torch.empty(4, 0, 33, device=DEV)
        out, last = ps.gated_recurrence(x, x, state=state, gating=gating)
        assert out.shape == x.shape and torch.equal(last, state)
        assert bool((ps.gated_recurrence(x, x, gating=gating)[1] == 0).all())
        c = ps.recurrence_carries(x)
        _, _, ds = ps.gated_recurrence_backward(x, x, x, c, dstate_out=state, gating=gating)
        assert torch.equal(ds, state)
        for shape in ((0, 7, 33), (2, 7, 0)):
            y = torch.empty(shape, device=DEV)
            out, last = ps.gated_recurrence(y, y, gating=gating)
            assert out.shape == y.shape and last.shape == (shape[0], shape[2])
        p = torch.full((9, 33), 3.0, device=DEV)
        none = torch.zeros(1, dtype=torch.int64, device=DEV)
        out = torch.full((9, 33), 5.0, device=DEV)
        _, last = ps.gated_recurrence(p, p, gating=gating, offsets=none, out=out)
        assert last.shape == (0, 33) and bool((out == 5.0).all())
        e = torch.empty(0, 33, device=DEV)
        five = torch.zeros(5, dtype=torch.int64, device=DEV)
        _, last = ps.gated_recurrence(e, e, state=state, gating=gating, offsets=five)
        assert torch.equal(last, state)


@pytest.mark.parametrize("dtype", TYPES)
def test_gates_at_the_ends_of_their_range(dtype):
    """Gates of the type's lowest and highest value, infinities and zeros: a is 0 or 1 exactly."""
    t = TYPES[dtype]
    big = torch.finfo(t).max
    r = rng(77)
    for gating, ends in (("sigmoid", [-big, big, float("inf"), float("-inf"), 0.0]), ("log", [-big, float("-inf"), 0.0]),
                         ("decay", [0.0, 1.0, -1.0])):
        shape = (2, 90, 64)
        x, dout = make(r, shape, t), make(r, shape, t)
        g = torch.tensor(r.choice(ends, shape)).to(t)
        state = make(r, (2, 64), torch.float32)
        a, _ = lo.decay(host(g), gating)
        assert set(np.unique(a)) <= {-1.0, 0.0, 0.5, 1.0}
        h, _, last = lo.recurrence(host(x), host(g), host(state), gating)
        size = np.abs(host(x)).cumsum(1) + np.abs(host(state))[:, None]
        gx, gg = x.to(DEV), g.to(DEV)
        c = ps.recurrence_carries(gx)
        out, state_out = ps.gated_recurrence(gx, gg, state=state.to(DEV), gating=gating, carries=c)
        close(out, h, size * 100 * lo.U, "h")  # at most 90 tokens' sums and 10 joins, each rounded once
        close(state_out, last, size[:, -1] * 100 * lo.U, "state")
        dx, dg, ds = ps.gated_recurrence_backward(dout.to(DEV), gx, gg, c, state=state.to(DEV), gating=gating)
        (wx, wg, ws), _ = lo.gradients(host(x), host(g), host(state), host(dout), None, gating)
        dsize = np.abs(host(dout))[:, ::-1].cumsum(1)[:, ::-1]
        close(dx, wx, dsize * 100 * lo.U, "dx")
        close(dg, wg, dsize * (size + np.abs(host(x))) * 250 * lo.U, "dgate")
        close(ds, ws, dsize[:, 0] * 100 * lo.U, "dstate")


def test_infinities_and_nan_stay_in_their_sequence():
    r = rng(5)
    lengths = [40, 100, 30, 1, 260, 7]
    off = torch.tensor(np.concatenate([[0], np.cumsum(lengths)])).to(DEV)
    n, d = sum(lengths), 65
    for bad in (float("inf"), float("nan")):
        x, g, dout = make(r, (n, d), torch.float32), gates(r, (n, d), "sigmoid", torch.float32), make(r, (n, d), torch.float32)
        state = make(r, (6, d), torch.float32)
        results = []
        for spoil in (False, True):
            y, e, s = x.clone(), dout.clone(), state.clone()
            if spoil:
                y[60], e[50], s[1], y[175], e[430] = bad, bad, bad, bad, bad
                g2 = g.clone()
                g2[130] = float("nan")
            else:
                g2 = g
            gx, gg = y.to(DEV), g2.to(DEV)
            c = ps.recurrence_carries(gx, off)
            out, last = ps.gated_recurrence(gx, gg, state=s.to(DEV), offsets=off, carries=c)
            dx, dg, ds = ps.gated_recurrence_backward(e.to(DEV), gx, gg, c, state=s.to(DEV), offsets=off)
            results.append((out, dx, dg, last, ds))
        clean = [0, 2, 3, 5]
        for a, b in zip(*results):
            for s in clean:
                rows = slice(int(off[s]), int(off[s + 1])) if a.shape[0] == n else slice(s, s + 1)
                assert torch.equal(a[rows], b[rows]) and bool(torch.isfinite(b[rows]).all())
        # and only what the formula reaches: the tokens before it are as they were
        assert torch.equal(results[0][0][170:175], results[1][0][170:175])
        assert not torch.isfinite(results[1][0][175]).any()


def test_gradient_against_differences():
    """The loss sum(h * p) + sum(state_out * q) along random directions of x, gate and state, in float64 by
    the oracle: (L(v + e) - L(v - e)) / 2 is right to e^2, and float32's part is far below 1e-3."""
    for gating in GATINGS:
        r = rng(31)
        shape, d = (2, 37, 5), 5
        x, g = make(r, shape, torch.float32), gates(r, shape, gating, torch.float32)
        state, p, q = make(r, (2, d), torch.float32), make(r, shape, torch.float32), make(r, (2, d), torch.float32)
        gx, gg = x.to(DEV), g.to(DEV)
        c = ps.recurrence_carries(gx)
        ps.gated_recurrence(gx, gg, state=state.to(DEV), gating=gating, carries=c)
        got = ps.gated_recurrence_backward(p.to(DEV), gx, gg, c, state=state.to(DEV), dstate_out=q.to(DEV), gating=gating)

        def loss(x, g, s):
            h, _, last = lo.recurrence(x, g, s, gating)
            return (h * host(p)).sum() + (last * host(q)).sum()

        for _ in range(4):
            v = [host(x), host(g), host(state)]
            w = [r.standard_normal(k.shape) for k in v]
            e = 1e-5
            diff = (loss(*[a + e * b for a, b in zip(v, w)]) - loss(*[a - e * b for a, b in zip(v, w)])) / (2 * e)
            along = sum((host(a) * b).sum() for a, b in zip(got, w))
            scale = sum(np.abs(host(a) * b).sum() for a, b in zip(got, w))
            assert abs(along - diff) <= 1e-5 * scale


@pytest.mark.parametrize("packed", [False, True])
def test_graph(packed):
    """Captured, replayed with other inputs in place, eager calls in between."""
    r = rng(8)
    d, s = 192, 3
    lengths = [500, 0, 700] if packed else [400] * 3
    shape = (1300, d) if packed else (3, 400, d)
    off = torch.tensor(np.concatenate([[0], np.cumsum(lengths)])).to(DEV) if packed else None
    x, g = (torch.zeros(shape, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dout, state = torch.zeros_like(x), torch.zeros(s, d, device=DEV)
    out, dx, dg = (torch.zeros_like(x) for _ in range(3))
    c = ps.recurrence_carries(x, off)

    def step():
        _, last = ps.gated_recurrence(x, g, state=state, offsets=off, out=out, carries=c)
        _, _, ds = ps.gated_recurrence_backward(dout, x, g, c, state=state, dstate_out=state, offsets=off, dx=dx, dgate=dg)
        return last, ds

    side = torch.cuda.Stream()
    for warm in (True, False):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            if warm:
                step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            kept = step()
        for turn in range(4):
            for t in (x, g, dout, state):
                t.copy_(torch.from_numpy(r.standard_normal(t.shape)).to(t.dtype))
            graph.replay()
            torch.cuda.synchronize()
            got = [v.clone() for v in (out, dx, dg, *kept)]
            want = step()
            torch.cuda.synchronize()
            for a, b in zip(got, (out, dx, dg, *want)):
                assert torch.equal(a, b)
    assert ps.workspace_error_flags(DEV) == 0


def test_two_streams_and_repeats():
    """Calls on two streams at once, many times over: the same bits."""
    r = rng(9)
    x, g = make(r, (2, 3000, 320), torch.bfloat16).to(DEV), gates(r, (2, 3000, 320), "sigmoid", torch.bfloat16).to(DEV)
    want = ps.gated_recurrence(x, g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(ps.gated_recurrence(x, g))
    torch.cuda.synchronize()
    for a in got:
        assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])
    for s in streams:
        assert ps.workspace_error_flags(DEV, s) == 0


@pytest.mark.parametrize("batch,channels", [(1, 64), (1, 512), (16, 2048), (64, 512), (520, 128)])
def test_many_tiles_and_chains(batch, channels):
    """Long sequences, and more chains of tiles than blocks that fit the GPU at once (a chain for each 128
    channels of each sequence): against the recurrence in float64 by doubling windows."""
    length = 20000 if batch == 1 else 1300
    g = torch.Generator(device=DEV).manual_seed(batch)
    x = torch.randn(batch, length, channels, device=DEV, generator=g).bfloat16()
    gate = (torch.randn(batch, length, channels, device=DEV, generator=g) + 1).bfloat16()
    c = ps.recurrence_carries(x)
    out, last = ps.gated_recurrence(x, gate, carries=c)
    dx, dg, ds = ps.gated_recurrence_backward(x, x, gate, c)

    def scan(a, b):
        step = 1
        while step < length:
            b = torch.cat([b[:, :step], b[:, step:] + a[:, step:] * b[:, :-step]], 1)
            a = torch.cat([a[:, :step], a[:, step:] * a[:, :-step]], 1)
            step *= 2
        return b

    for s in range(0, batch, max(1, batch // 4)):
        xs, a = x[s:s + 1].double(), torch.sigmoid(gate[s:s + 1].double())
        h = scan(a, (1 - a) * xs)
        # decays are below 0.995 (gates below 5.3), so what float32 rounds away is some (10 + 6) * 200 * 2^-24 =
        # 2e-4 of |h| < 6 or lambda < 50 at the very worst; 2^-8 of a value is bfloat16's rounding (2^-9) and more
        assert bool(((out[s:s + 1].double() - h).abs() <= h.abs() * 2.0**-8 + 1e-3).all())
        assert bool(((last[s] - h[0, -1]).abs() <= 1e-3).all())
        behind = torch.cat([torch.zeros_like(a[:, :1]), a.flip(1)[:, :-1]], 1)
        lam = scan(behind, xs.flip(1)).flip(1)
        before = torch.cat([torch.zeros_like(h[:, :1]), h[:, :-1]], 1)
        want = lam * (1 - a)
        assert bool(((dx[s:s + 1].double() - want).abs() <= want.abs() * 2.0**-8 + 1e-3).all())
        want = lam * (before - xs) * a * (1 - a)
        assert bool(((dg[s:s + 1].double() - want).abs() <= want.abs() * 2.0**-8 + 1e-2).all())
        assert bool(((ds[s] - (a * lam)[0, 0]).abs() <= 1e-2).all())
    again = ps.gated_recurrence(x, gate)[0]
    assert torch.equal(again, out) and ps.workspace_error_flags(DEV) == 0


def test_refused_by_the_binding():
    x = torch.zeros(2, 5, 8, device=DEV)
    with pytest.raises(ValueError):
        ps.gated_recurrence(x, x, gating="tanh")
    with pytest.raises(ValueError):
        ps.gated_recurrence(x, x[:, :4])
    with pytest.raises(ValueError):
        ps.gated_recurrence(x, x.half())
    with pytest.raises(TypeError):
        ps.gated_recurrence(x.double(), x.double())
    with pytest.raises(ValueError):
        ps.gated_recurrence(x, x.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError):
        ps.gated_recurrence(x, x, state=torch.zeros(2, 8, device=DEV, dtype=torch.float16))
    with pytest.raises(ValueError):
        ps.gated_recurrence(x, x, carries=torch.zeros(3, 8, device=DEV))
    with pytest.raises(ps.LibscanError):
        ps.gated_recurrence(x, x, out=x)
    with pytest.raises(ps.LibscanError):
        ps.gated_recurrence(x, x, out=torch.zeros(1, 5, 8, device=DEV).expand(2, 5, 8))
    with pytest.raises(ValueError):
        ps.gated_recurrence(x, x, offsets=torch.zeros(3, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        ps.gated_recurrence(x[0], x[0], offsets=torch.zeros(3, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        ps.gated_recurrence_backward(x, x, x, None)
    with pytest.raises(ValueError):
        ps.gated_recurrence(x.cpu(), x.cpu())
