"""experts_sort, experts_gather, experts_combine and its gradients against the oracle."""
import numpy as np
import pytest
import torch

import layer_oracle as lo
import prefix_scan_stream_amd as ps

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def rng(seed):
    return np.random.default_rng(20260925 + seed)


def host(t):
    return t.double().cpu().numpy()


def sort_check(experts, num_experts, dtype):
    e = torch.from_numpy(experts).to(dtype).to(DEV)
    offsets, order, places = ps.experts_sort(e, num_experts)
    want = lo.sort(experts, num_experts)
    for got, w in zip((offsets, order, places), want):
        assert np.array_equal(got.cpu().numpy(), w)


SIZES = [0, 1, 2, 63, 64, 65, 511, 512, 513, 4095, 4096, 4097, 8193, 30000, 131072, 600001]


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64], ids=str)
@pytest.mark.parametrize("n", SIZES)
def test_sort_sizes(n, dtype):
    r = rng(n)
    for num in ((1, 8, 255) if n < 100000 else (64,)):
        e = r.integers(0, num, n)
        if num > 1:
            e[r.random(n) < 0.1] = -1
        sort_check(e, num, dtype)


@pytest.mark.parametrize("num", [1, 2, 3, 63, 64, 65, 127, 128, 256, 511, 512, 513, 1000, 1024])
def test_sort_experts(num):
    r = rng(num)
    for n in (40, 5000, 20000):
        sort_check(r.integers(0, num, n).reshape(-1, 4), num, torch.int64)
        sort_check(r.integers(-2, num + 3, n).reshape(-1, 2), num, torch.int32)  # some nowhere
    sort_check(np.full(9000, num - 1), num, torch.int32)  # all to one expert
    sort_check(np.full(9000, -1), num, torch.int32)
    sort_check(np.sort(r.integers(0, num, 9000))[::-1].copy(), num, torch.int64)


def test_sort_numbers_far_out():
    e = np.array([3, 2**40, -(2**62), 2**32 + 1, 1, -1, 7, 8, 2**63 - 1], dtype=np.int64)
    sort_check(e, 8, torch.int64)
    sort_check(np.array([3, 2**31 - 1, -(2**31), 1], dtype=np.int64), 8, torch.int32)


def routing(r, tokens, top, num, dropped):
    e = np.stack([r.permutation(num)[:top] for _ in range(tokens)]) if tokens and top else np.zeros((tokens, top), dtype=np.int64)
    e[r.random(e.shape) < dropped] = -1
    return lo.sort(e, num)[2]


SHAPES = [(1, 1, 1), (1, 8, 64), (3, 2, 1), (5, 3, 65), (17, 8, 512), (61, 6, 1000), (33, 9, 513), (130, 4, 2048), (40, 17, 96),
          (7, 1, 4100), (0, 3, 64), (4, 0, 64), (4, 2, 0), (9, 8, 8200)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_moves(dtype, shape):
    tokens, top, d = shape
    t = TYPES[dtype]
    half = torch.finfo(t).eps / 2
    for case in range(4):
        r = rng(sum(shape) * 10 + case)
        places = routing(r, tokens, top, max(top, 20), 0.2 if case % 2 else 0.0)
        pairs = tokens * top
        gp = torch.from_numpy(places.astype(np.int32)).to(DEV)
        num_rows = pairs if case < 2 else max(1, pairs // 2)  # places past the rows take part in nothing

        def mat(rows, extra=0):
            big = torch.from_numpy(r.standard_normal((rows, d + extra))).to(t).to(DEV)
            return big[:, extra:]

        odd = 3 if case == 3 else 0  # rows at odd elements
        x, rows = mat(tokens, odd), mat(num_rows, odd)
        buf = torch.full((num_rows, d + odd), 9.0, dtype=t, device=DEV)[:, odd:]
        got = ps.experts_gather(x, gp, out=buf)
        assert np.array_equal(host(got), lo.gather(host(x), places, np.full((num_rows, d), 9.0)))

        for wtype in (None, torch.float32, t):
            w = None if wtype is None else torch.from_numpy(r.standard_normal((tokens, top))).to(wtype).to(DEV)
            want, size = lo.combine(host(rows), places, None if w is None else host(w))
            got = ps.experts_combine(rows, gp, w)
            # a product and an addition a pair in float32, one rounding at the end
            room = size * top * 2 * lo.U * (1 + half) + np.abs(want) * half + torch.finfo(t).smallest_normal * half * 2
            assert (np.abs(host(got) - want) <= room).all()
            if w is None:
                continue
            drows = torch.full((num_rows, d), 9.0, dtype=t, device=DEV)
            dout = mat(tokens, odd)
            drows, dw = ps.experts_combine_backward(dout, rows, gp, w, drows=drows)
            wr, ww, wsize = lo.combine_backward(host(dout), host(rows), places, host(w), np.full((num_rows, d), 9.0))
            assert (np.abs(host(drows) - wr) <= np.abs(wr) * (half * (1 + lo.U) + lo.U) + torch.finfo(t).smallest_normal * half * 2).all()
            whalf = torch.finfo(wtype).eps / 2
            # each lane adds up to d / 64 + 8 products, the lanes' sums meet in 6 steps (more at element width)
            steps = d + 8
            room = wsize * steps * lo.U * (1 + whalf) + np.abs(ww) * whalf + torch.finfo(wtype).smallest_normal * whalf * 2
            assert (np.abs(host(dw) - ww) <= room).all()


def test_pairs_without_a_row_are_not_read():
    """NaN weights and NaN rows of pairs that go nowhere stay out; a token with no row gets zeros."""
    places = torch.tensor([[0, -1], [-1, -1], [1, 5]], dtype=torch.int32, device=DEV)
    nan = float("nan")
    w = torch.tensor([[2.0, nan], [nan, float("inf")], [0.5, nan]], device=DEV)
    rows = torch.stack([torch.arange(8.0), torch.ones(8), torch.full((8,), nan)]).to(DEV)
    out = ps.experts_combine(rows, places, w)
    assert out.tolist() == [[2.0 * i for i in range(8)], [0.0] * 8, [0.5] * 8]
    dout = torch.ones(3, 8, device=DEV)
    drows, dw = ps.experts_combine_backward(dout, rows, places, w, drows=torch.full((3, 8), -1.0, device=DEV))
    assert dw.tolist() == [[28.0, 0.0], [0.0, 0.0], [8.0, 0.0]]
    assert drows.tolist() == [[2.0] * 8, [0.5] * 8, [-1.0] * 8]


def test_one_choice_a_token_as_a_vector():
    e = torch.tensor([2, 0, 2, 1], device=DEV)
    offsets, order, places = ps.experts_sort(e, 3)
    assert places.tolist() == [2, 0, 3, 1] and order.tolist() == [1, 3, 0, 2] and offsets.tolist() == [0, 1, 2, 4]
    x = torch.arange(8.0, device=DEV).reshape(4, 2)
    rows = ps.experts_gather(x, places)
    assert rows.tolist() == x[order.long()].tolist()
    assert torch.equal(ps.experts_combine(rows, places), x)


def test_graph():
    """Sort, gather, combine and gradients captured together; replays against eager calls."""
    r = rng(3)
    tokens, top, num, d = 3000, 4, 40, 320
    e = torch.zeros(tokens, top, dtype=torch.int64, device=DEV)
    x, dout = (torch.zeros(tokens, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    w = torch.zeros(tokens, top, device=DEV)
    rows = torch.zeros(tokens * top, d, dtype=torch.bfloat16, device=DEV)
    drows = torch.zeros_like(rows)

    def step():
        offsets, order, places = ps.experts_sort(e, num)
        ps.experts_gather(x, places, out=rows)
        out = ps.experts_combine(rows, places, w)
        _, dw = ps.experts_combine_backward(dout, rows, places, w, drows=drows)
        return offsets, order, places, out, dw, ps.experts_combine(drows, places)

    side = torch.cuda.Stream()
    for warm in (True, False):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            if warm:
                step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            kept = step()
        for _ in range(4):
            e.copy_(torch.from_numpy(r.integers(-1, num, (tokens, top))))
            for t in (x, dout, w):
                t.copy_(torch.from_numpy(r.standard_normal(t.shape)).to(t.dtype))
            rows.zero_(), drows.zero_()
            graph.replay()
            torch.cuda.synchronize()
            got = [v.clone() for v in (*kept, rows, drows)]
            rows.zero_(), drows.zero_()
            want = step()
            for a, b in zip(got, (*want, rows, drows)):
                assert torch.equal(a, b)


def test_refused_by_the_binding():
    e = torch.zeros(4, 2, dtype=torch.int64, device=DEV)
    p = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    x, rows = torch.zeros(4, 8, device=DEV), torch.zeros(8, 8, device=DEV)
    w = torch.ones(4, 2, device=DEV)
    for bad in (lambda: ps.experts_sort(e.float(), 3), lambda: ps.experts_gather(x.double(), p),
                lambda: ps.experts_combine_backward(x, rows, p, w, dweights=w.half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ps.experts_sort(e.t(), 3), lambda: ps.experts_sort(e, 3, order=torch.zeros(7, dtype=torch.int32, device=DEV)),
                lambda: ps.experts_gather(x, p[:3]), lambda: ps.experts_gather(x, p.long()),
                lambda: ps.experts_combine(rows, p, w[:3]), lambda: ps.experts_combine_backward(x, rows.half(), p, w),
                lambda: ps.experts_combine_backward(x, rows, p, None), lambda: ps.experts_sort(e.cpu(), 3),
                lambda: ps.experts_combine(rows.t(), p)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ps.experts_sort(e, 0), lambda: ps.experts_sort(e, 1025), lambda: ps.experts_gather(rows, torch.zeros(8, 1, dtype=torch.int32, device=DEV), out=rows),
                lambda: ps.experts_combine(rows, p, w, out=rows[:4])):
        with pytest.raises(ps.LibscanError):
            bad()
