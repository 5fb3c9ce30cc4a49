"""The gated recurrence and the experts' calls at their limits: waits that run out, graphs that share a
stream, host threads, indexes past 32 bits, more sequences and tokens than one launch holds."""
import ctypes
import os
import threading

import pytest
import torch

import prefix_scan_stream_amd as ps

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
SPIN = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "prefix_scan_stream_amd", "libscan_spin1.so")


def rand(*shape, seed=0, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, device=DEV, generator=g).to(dtype)


def test_waits_that_run_out_are_reported():
    """libscan_spin1.so ends every wait at its first empty poll: a call of many tiles says so, stays inside its
    buffers, and the workspace is good again once it is initialised."""
    if not os.path.exists(SPIN):
        pytest.fail(f"{SPIN} is missing: run __graft_entry__.build() first")
    normal = ps.load_library()
    spin = ctypes.CDLL(SPIN)
    for name in ("gated_recurrence", "gated_recurrence_backward", "ls_recurrence_workspace_bytes", "ls_workspace_init", "ls_workspace_check"):
        getattr(spin, name).argtypes = getattr(normal, name).argtypes
    length, d = 30000, 64
    x, gate = rand(1, length, d), rand(1, length, d, seed=1)
    want, last = ps.gated_recurrence(x, gate)
    size = ctypes.c_size_t(0)
    assert normal.ls_recurrence_workspace_bytes(1, length, d, 0, 2, ctypes.byref(size)) == 0 and size.value > 256
    ws = torch.empty(size.value + 256, dtype=torch.uint8, device=DEV)
    ws[size.value:] = 77
    stream = torch.cuda.current_stream(DEV).cuda_stream
    guarded = torch.full((length + 2, d), 5.0, dtype=torch.bfloat16, device=DEV)
    out, state = guarded[1:-1], torch.full((3, d), 5.0, device=DEV)
    flags = ctypes.c_uint32(0)
    n = (size.value + 15) // 16 * 16

    def call(lib):
        assert lib.gated_recurrence(x.data_ptr(), length * d, d, gate.data_ptr(), length * d, d, out.data_ptr(), length * d, d,
                                    None, d, state[1].data_ptr(), d, None, None, 1, length, d, 2, 2, ws.data_ptr(), size.value,
                                    stream) == 0
        return lib.ls_workspace_check(ws.data_ptr(), ctypes.byref(flags), stream)

    assert normal.ls_workspace_init(ws.data_ptr(), n, stream) == 0
    assert call(spin) == ps.LS_ERR_INCOMPLETE and flags.value == 1
    assert bool((guarded[0] == 5.0).all()) and bool((guarded[-1] == 5.0).all()) and bool((ws[n:] == 77).all())
    assert bool((state[0] == 5.0).all()) and bool((state[2] == 5.0).all())
    assert normal.ls_workspace_init(ws.data_ptr(), n, stream) == 0
    for _ in range(3):
        assert call(normal) == ps.LS_OK and flags.value == 0
        assert torch.equal(out, want[0]) and torch.equal(state[1], last[0])


def work_of(size, seed):
    x, gate = rand(2, size, 192, seed=seed), rand(2, size, 192, seed=seed + 1)
    packed = torch.tensor([0, size // 3, size // 3, size], device=DEV)
    experts = torch.randint(-1, 30, (size, 4), device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed))
    state = rand(2, 192, seed=seed + 2, dtype=torch.float32)

    def work():
        c = ps.recurrence_carries(x)
        out, last = ps.gated_recurrence(x, gate, state=state, carries=c)
        back = ps.gated_recurrence_backward(out, x, gate, c, state=state)
        return [out, last, *back, ps.gated_recurrence(x[0], gate[0], offsets=packed)[0], *ps.experts_sort(experts, 30)]
    return work


def test_graphs_in_any_order():
    works = [work_of(size, 10 * size) for size in (3000, 1700, 2500)]
    wants = [[v.clone() for v in w()] for w in works]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        works[0]()
    torch.cuda.synchronize()
    graphs = []
    for w in works:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kept = w()
        graphs.append((graph, kept))
    for turn in ((0, 1, 2), (2, 0, 0, 1), (1, 1, 2, 0)):
        for i in turn:
            for v in graphs[i][1]:
                v.zero_()
            graphs[i][0].replay()
            with torch.cuda.stream(side):
                eager = works[(i + 1) % 3]()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(graphs[i][1], wants[i]))
            assert all(torch.equal(a, b) for a, b in zip(eager, wants[(i + 1) % 3]))
    # beside each other, on streams of their own
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(5):
        for (graph, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, kept), want in zip(graphs, wants):
        assert all(torch.equal(a, b) for a, b in zip(kept, want))


def test_threads_on_one_stream():
    works = [work_of(size, size) for size in (2000, 900, 1500, 40)]
    wants = [[v.clone() for v in w()] for w in works]
    torch.cuda.synchronize()
    wrong = []

    def go(i):
        for _ in range(15):
            got = works[i]()
            torch.cuda.current_stream().synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, wants[i])):
                wrong.append(i)

    threads = [threading.Thread(target=go, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_more_chains_than_blocks_on_three_streams():
    """More blocks that wait than the GPU holds, from calls beside each other: all of them end."""
    data = [(rand(40, 400, 768, seed=i), rand(40, 400, 768, seed=9 + i)) for i in range(3)]
    wants = [ps.gated_recurrence(x, g)[0].clone() for x, g in data]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in data]
    for _ in range(6):
        got = []
        for s, (x, g) in zip(streams, data):
            with torch.cuda.stream(s):
                got.append(ps.gated_recurrence(x, g)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, wants))
    assert all(ps.workspace_error_flags(DEV, s) == 0 for s in streams)


def test_elements_past_32_bits():
    """A sequence of more than 2^31 elements: its end is as of the last 4000 tokens alone (decays below 0.9
    leave nothing of what was before them after 1000: 0.9^1000 < 2^-150), and so are the gradients at its start."""
    d, length = 2048, (1 << 20) + 3000
    x = torch.empty(1, length, d, dtype=torch.bfloat16, device=DEV)
    for r in range(0, length, 1 << 17):
        x[:, r:r + (1 << 17)] = rand(1, min(1 << 17, length - r), d, seed=r)
    gate = x.clamp_max(2.0)
    c = ps.recurrence_carries(x)
    out, last = ps.gated_recurrence(x, gate, carries=c)
    tail, tail_last = ps.gated_recurrence(x[:, -4032:], gate[:, -4032:])
    assert torch.allclose(out[:, -2000:].float(), tail[:, -2000:].float(), rtol=2.0**-7, atol=1e-5)
    assert torch.allclose(last, tail_last, rtol=1e-5, atol=1e-6)
    dx, dg, ds = ps.gated_recurrence_backward(out, x, gate, c)
    hc = ps.recurrence_carries(x[:, :4000])
    ps.gated_recurrence(x[:, :4000], gate[:, :4000], carries=hc)
    hx, hg, hs = ps.gated_recurrence_backward(out[:, :4000], x[:, :4000], gate[:, :4000], hc)
    for a, b in ((dx, hx), (dg, hg)):
        assert torch.allclose(a[:, :2000].float(), b[:, :2000].float(), rtol=2.0**-7, atol=1e-5)
    assert torch.allclose(ds, hs, rtol=1e-5, atol=1e-6)
    assert bool(torch.isfinite(dx[:, -1]).all()) and ps.workspace_error_flags(DEV) == 0


def test_rows_past_32_bits():
    tokens, top, d = 150000, 4, 4096
    assert tokens * top * d > 1 << 31
    x = rand(tokens, d)
    experts = torch.randint(0, 64, (tokens, top), device=DEV, generator=torch.Generator(device=DEV).manual_seed(1))
    offsets, order, places = ps.experts_sort(experts, 64)
    rows = ps.experts_gather(x, places)
    some = torch.cat([torch.arange(0, tokens * top, 997, device=DEV), torch.arange(tokens * top - 5, tokens * top, device=DEV)])
    assert torch.equal(rows[some], x[order[some].long() // top])
    weights = torch.rand(tokens, top, device=DEV)
    out = ps.experts_combine(rows, places, weights)
    at = some[some < tokens]
    want = x[at].double() * weights[at].double().sum(1, keepdim=True)
    # the four products are of one value each: three additions and a rounding
    assert bool(((out[at].double() - want).abs() <= want.abs() * (2.0**-8 + 2.0**-20) + 1e-30).all())
    drows, dweights = ps.experts_combine_backward(x, rows, places, weights, drows=rows.clone())
    p = order[some].long()
    want = x[p // top].double() * weights.reshape(-1)[p].double()[:, None]
    assert bool(((drows[some].double() - want).abs() <= want.abs() * (2.0**-8 + 2.0**-20) + 1e-30).all())
    want = (x[at].double() ** 2).sum(1, keepdim=True).expand(-1, top)
    assert bool(((dweights[at].double() - want).abs() <= want * d * 2.0**-24).all())


def test_more_sequences_than_a_launch_holds():
    batch = (1 << 22) + 1001
    x, gate = rand(batch, 2, 2), rand(batch, 2, 2, seed=1)
    state = rand(batch, 2, seed=2, dtype=torch.float32)
    c = ps.recurrence_carries(x)
    out, last = ps.gated_recurrence(x, gate, state=state, carries=c)
    dx, dg, ds = ps.gated_recurrence_backward(x, x, gate, c, state=state)
    xs, a = x.double(), torch.sigmoid(gate.double())
    h0 = state.double()
    h1 = a[:, 0] * h0 + (1 - a[:, 0]) * xs[:, 0]
    h2 = a[:, 1] * h1 + (1 - a[:, 1]) * xs[:, 1]
    l2 = xs[:, 1]
    l1 = xs[:, 0] + a[:, 1] * l2
    near = lambda got, want: bool(((got.double() - want).abs() <= want.abs() * 2.0**-8 + 1e-5).all())
    assert near(out[:, 0], h1) and near(out[:, 1], h2) and near(last, h2)
    assert near(dx[:, 1], l2 * (1 - a[:, 1])) and near(dx[:, 0], l1 * (1 - a[:, 0])) and near(ds, l1 * a[:, 0])
    assert near(dg[:, 1], l2 * (h1 - xs[:, 1]) * a[:, 1] * (1 - a[:, 1]))


@pytest.mark.parametrize("extra", [1, 1001])
def test_more_long_sequences_than_a_launch_holds(extra):
    """Sequences of several tiles: those of the second launch walk as the first's do, and take nothing of the
    workspace, which is none."""
    batch, length = (1 << 22) + extra, 130
    x, gate = rand(1, length, 1).expand(batch, -1, -1), rand(1, length, 1, seed=1).expand(batch, -1, -1)
    size = ctypes.c_size_t(0)
    assert ps.load_library().ls_recurrence_workspace_bytes(batch, length, 1, 0, 2, ctypes.byref(size)) == 0 and size.value <= 256
    c = ps.recurrence_carries(x)
    out, last = ps.gated_recurrence(x, gate, carries=c)
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(last, last[:1].expand_as(last))
    h, want = 0.0, []
    for xt, gt in zip(x[0, :, 0].double().tolist(), torch.sigmoid(gate[0, :, 0].double()).tolist()):
        h = gt * h + (1 - gt) * xt
        want.append(h)
    want = torch.tensor(want, device=DEV, dtype=torch.float64)
    # 2^-8 of the rounding to bfloat16, 1e-5 for 130 steps in float32 (values up to 4)
    assert bool(((out[0, :, 0].double() - want).abs() <= want.abs() * 2.0**-8 + 1e-5).all())
    dx, dg, ds = ps.gated_recurrence_backward(x, x, gate, c)
    one = ps.gated_recurrence_backward(x[:512], x[:512], gate[:512], c[: 512 * 3])
    for got, few in zip((dx, dg, ds), one):
        assert torch.equal(got, few[:1].expand_as(got))


def test_nan_of_any_bits_stays_in_its_channel():
    """float32 gates may be NaN of any bits, those of the kernels' own marks among them."""
    length, d = 4000, 64
    x, gate = rand(1, length, d, dtype=torch.float32), torch.sigmoid(rand(1, length, d, seed=1, dtype=torch.float32))
    want = ps.gated_recurrence(x, gate, gating="decay")
    bits = gate.clone().view(torch.int32)
    bits[0, 500, 0], bits[0, 2500, 0] = 0x7FC0C0DE, 0x7FC0C0DE
    out, last = ps.gated_recurrence(x, bits.view(torch.float32), gating="decay")
    assert torch.equal(out[:, :, 1:], want[0][:, :, 1:]) and torch.equal(last[:, 1:], want[1][:, 1:])
    assert torch.equal(out[0, :500, 0], want[0][0, :500, 0]) and bool(out[0, 500:, 0].isnan().all())


def test_more_tokens_than_blocks():
    tokens = (1 << 25) + 77  # 32 tokens of 8 channels a block, 2^20 blocks
    x = torch.arange(tokens, device=DEV, dtype=torch.int32)[:, None].expand(tokens, 8).to(torch.bfloat16)
    places = torch.arange(tokens - 1, -1, -1, device=DEV, dtype=torch.int32)[:, None]
    rows = ps.experts_gather(x, places)
    assert torch.equal(rows, x.flip(0))
    back = ps.experts_combine(rows, places)
    assert torch.equal(back, x)
    weights = torch.full((tokens, 1), 2.0, device=DEV)
    drows, dw = ps.experts_combine_backward(torch.ones_like(x), rows, places, weights)
    assert bool((drows == 2.0).all()) and torch.equal(dw[:, 0], 8 * x[:, 0].float())


@pytest.mark.parametrize("top", [1, 2, 3, 4, 5, 8, 11])
@pytest.mark.parametrize("mib", [40, 72, 300])
def test_many_rows(mib, top):
    """Few rows, more than the near caches hold and more than all caches hold move by different loads and stores,
    which change no value: the rows and sums of some tokens are those of these tokens alone."""
    d = 1032
    tokens = (mib << 20) // (2 * d * top) + 3
    x, rows = rand(tokens, d), rand(tokens * top, d, seed=1)
    gen = torch.Generator(device=DEV).manual_seed(2)
    places = torch.randperm(tokens * top, device=DEV, generator=gen).view(tokens, top).to(torch.int32)
    places[5::97, 0] = -1
    weights = torch.rand(tokens, top, device=DEV, generator=gen)
    some = torch.cat([torch.arange(40, device=DEV), torch.randint(0, tokens, (200,), device=DEV, generator=gen).unique(),
                      torch.arange(tokens - 40, tokens, device=DEV)]).unique()
    held = places >= 0

    drows = torch.full_like(rows, 7.0)
    got = ps.experts_gather(x, places, out=drows)
    assert torch.equal(got[places[held].long()], x[held.nonzero()[:, 0]])
    untouched = torch.ones(tokens * top, dtype=torch.bool, device=DEV)
    untouched[places[held].long()] = False
    assert bool((got[untouched] == 7.0).all())

    sums = ps.experts_combine(rows, places, weights)
    assert torch.equal(sums[some], ps.experts_combine(rows, places[some], weights[some]))
    at = places[some].long().clamp(min=0)
    w = torch.where(held[some], weights[some], 0).double()
    parts = rows[at].double() * w[..., None]
    # a sum of `top` products in float32, rounded to bfloat16
    bound = parts.abs().sum(1) * (top + 1) * 2.0**-24 + (parts.sum(1).abs() * (1 + 2.0**-20) + 2.0**-133) * 2.0**-8
    assert bool(((sums[some].double() - parts.sum(1)).abs() <= bound).all())

    drows.fill_(7.0)
    drows, dweights = ps.experts_combine_backward(x, rows, places, weights, drows=drows)
    few, few_weights = ps.experts_combine_backward(x[some], rows, places[some], weights[some], drows=torch.full_like(rows, 7.0))
    named = places[some][held[some]].long()
    assert torch.equal(drows[named], few[named]) and torch.equal(dweights[some], few_weights)
    assert bool((drows[untouched] == 7.0).all())
    exact = (weights[some].double()[..., None] * x[some].double()[:, None])[held[some]]
    # one product in float32, rounded to bfloat16
    assert bool(((drows[named].double() - exact).abs() <= exact.abs() * (2.0**-8 + 2.0**-23) + 2.0**-133).all())
    dots = x[some].double()[:, None] * rows[at].double()
    wrong = (dweights[some].double() - torch.where(held[some], dots.sum(2), 0)).abs()
    assert bool((wrong <= dots.abs().sum(2) * (d + 1) * 2.0**-24).all())


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("gating", ["sigmoid", "log", "decay"])
@pytest.mark.parametrize("dtype, d", [(torch.float32, 129), (torch.float16, 258), (torch.bfloat16, 259), (torch.float32, 325),
                                      (torch.float16, 643), (torch.bfloat16, 1282)], ids=str)
def test_many_tokens(dtype, d, gating, packed):
    """Tokens that fill the caches are loaded by other loads than fewer, which changes no value: two halves of a
    call, tile by tile the same work, give what the call gives."""
    half = -(-(60 << 20) // (2 * d * dtype.itemsize)) // 1024 * 1024 + 1024
    x, gate, dout = (rand(2, half, d, seed=i, dtype=dtype) for i in range(3))
    if gating != "sigmoid":
        gate = torch.sigmoid(gate.float()).to(dtype) if gating == "decay" else -gate.abs()
    state, dstate = rand(2, d, seed=3, dtype=torch.float32), rand(2, d, seed=4, dtype=torch.float32)

    def call(x, gate, dout, state, dstate):
        n, offsets = x.shape[0], None
        if packed:
            offsets = torch.arange(n + 1, device=DEV) * half
            x, gate, dout = (t.reshape(-1, d) for t in (x, gate, dout))
        carries = ps.recurrence_carries(x, offsets)
        out, last = ps.gated_recurrence(x, gate, state, gating, offsets=offsets, carries=carries)
        grads = ps.gated_recurrence_backward(dout, x, gate, carries, state=state, dstate_out=dstate, gating=gating, offsets=offsets)
        return [t.reshape(n, -1) for t in (out, last, *grads)]

    whole = call(x, gate, dout, state, dstate)
    parts = [call(x[i:i + 1], gate[i:i + 1], dout[i:i + 1], state[i:i + 1], dstate[i:i + 1]) for i in range(2)]
    for got, *want in zip(whole, *parts):
        assert torch.equal(got, torch.cat(want)) and bool(torch.isfinite(got).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
def test_a_token_each_with_states_off_32_bytes(dtype):
    """States and carries at 16 bytes past a border of 32, with rows an odd multiple of 16 bytes apart."""
    batch, d = 37, 264
    x, gate = rand(batch, d, dtype=dtype), rand(batch, d, seed=1, dtype=dtype)
    state = rand(batch, d, seed=2, dtype=torch.float32)
    kept = ps.recurrence_carries(x)
    want = ps.gated_recurrence(x, gate, state=state, carries=kept)

    def off(columns):
        flat = torch.full((batch * columns + 8,), 5.0, device=DEV)
        first = (16 - flat.data_ptr() % 32) % 32 // 4
        return flat, flat[first:first + batch * columns].view(batch, columns)

    (_, before), (_, after), (flat, carries) = off(d + 4), off(d + 4), off(d)
    for t in (before, after, carries):
        assert t.data_ptr() % 32 == 16
    before[:, :d] = state
    out, last = ps.gated_recurrence(x, gate, state=before[:, :d], state_out=after[:, :d], carries=carries)
    assert torch.equal(out, want[0]) and torch.equal(last, want[1]) and torch.equal(carries, kept)
    assert bool((after[:, d:] == 5.0).all()) and int((flat == 5.0).sum()) >= 8
    out, last = ps.gated_recurrence(x, gate, state=before[:, :d], state_out=before[:, :d])  # in place
    assert torch.equal(out, want[0]) and torch.equal(last, want[1])


@pytest.mark.parametrize("d", [2, 65, 700])
def test_empty_sequences_in_any_number(d):
    """Hundreds of thousands of empty sequences in front of, between and behind others change nothing for these, and
    hand on their states."""
    lengths = [0] * 200000 + [50] + [0] * 9000 + [300] + [0] * 300000 + [1, 0, 2] + [0] * 8192 + [90] + [0] * 100000
    lens = torch.tensor(lengths, device=DEV)
    offsets = torch.cat([lens.new_zeros(1), lens.cumsum(0)])
    held, empty = (lens > 0).nonzero()[:, 0], lens == 0
    n = int(offsets[-1])
    x, gate, dout = (rand(n, d, seed=i) for i in range(3))
    state, dstate = (rand(len(lengths), d, seed=3 + i, dtype=torch.float32) for i in range(2))

    def call(offsets, state, dstate):
        carries = ps.recurrence_carries(x, offsets)
        out, last = ps.gated_recurrence(x, gate, state, offsets=offsets, carries=carries)
        return [out, *ps.gated_recurrence_backward(dout, x, gate, carries, state=state, dstate_out=dstate, offsets=offsets), last]

    out, dx, dgate, ds, last = call(offsets, state, dstate)
    few = call(torch.cat([offsets[:1], offsets[held + 1]]), state[held], dstate[held])
    for got, want in zip((out, dx, dgate, ds[held], last[held]), few):
        assert torch.equal(got, want)
    assert torch.equal(last[empty], state[empty]) and torch.equal(ds[empty], dstate[empty])
    assert ps.workspace_error_flags(DEV) == 0
