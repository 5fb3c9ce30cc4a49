"""pages_append, slot_map and pages_release against the oracle, entry by entry."""
import numpy as np
import pytest
import torch

import decode_oracle as do
import prefix_scan_stream_amd as ps
from gpu_util import DEV, to_dev, to_host

pytestmark = pytest.mark.gpu

# one chunk of the scan holds 4096 requests; a turn of outputs 2048
REQUESTS = [0, 1, 2, 63, 256, 700, 4095, 4096, 4097, 9001]


def make(requests, page, longest, new, columns, seed, pool=None):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, requests).astype(np.int32)
    add = rng.integers(0, new + 1, requests).astype(np.int32)
    add[rng.random(requests) < 0.2] = 0
    held = -(-lens // page)
    tables = np.full((requests, columns), -1, dtype=np.int32)
    pool = max(1, requests * columns) if pool is None else pool
    pages = rng.permutation(max(pool, int(held.sum())))
    at = 0
    for r in range(requests):
        n = min(int(held[r]), columns)
        tables[r, :n] = pages[at:at + n]
        at += n
    free = np.full(len(pages), -1, dtype=np.int32)
    free[:len(pages) - at] = pages[at:]
    return lens, add, tables, free, len(pages) - at


def check_append(lens, add, tables, free, count, page, stride=None):
    want = do.append(lens, add, tables, free, count, page)
    t = to_dev(tables)
    if stride:
        wide = torch.full((tables.shape[0], stride), -9, dtype=torch.int32, device=DEV)
        wide[:, :tables.shape[1]] = t
        t = wide[:, :tables.shape[1]]
    left, granted = ps.pages_append(to_dev(lens), to_dev(add), t, to_dev(free),
                                    torch.tensor([count], device=DEV), page)
    assert np.array_equal(to_host(t), want[0])
    assert np.array_equal(to_host(granted), want[1])
    assert int(to_host(left)[0]) == want[2]
    if stride:
        assert bool((wide[:, tables.shape[1]:] == -9).all())


@pytest.mark.parametrize("page", [1, 16, 24])
@pytest.mark.parametrize("requests", REQUESTS)
def test_append(requests, page):
    print(f"append requests={requests} page={page}", flush=True)
    case = make(requests, page, 10 * page, 5 * page, 17, 40 + requests)
    check_append(*case, page)
    # the list runs out half way; the table's rows lie apart
    lens, add, tables, free, count = case
    asked = int((-(-(lens + add) // page) - -(-lens // page)).sum())
    check_append(lens, add, tables, free, min(count, asked // 2), page, stride=20)
    # some requests do not fit the table
    check_append(lens, add, tables[:, :9].copy(), free, count, page)


def test_append_corner_values():
    top = 2**31 - 1
    lens = np.array([-5, 0, top, top, 0, 3, top - 1], dtype=np.int32)
    add = np.array([3, -7, 1, top, top, 0, 1], dtype=np.int32)
    tables = np.full((7, 6), -1, dtype=np.int32)
    free = np.arange(100, dtype=np.int32)
    for page in (1, 2, 1 << 20, 1 << 29, 1 << 30, (1 << 30) + 1, top):
        print(f"page={page}", flush=True)
        check_append(lens, add, tables, free, 100, page)
    check_append(lens, add, tables, free, -3, 1 << 30)       # no fewer than none free
    check_append(lens, add, tables, free[:1], 50, 1 << 30)   # no more than the list holds
    check_append(lens, add, np.zeros((7, 0), dtype=np.int32), free, 100, 16)
    check_append(lens, add, tables, np.zeros(0, dtype=np.int32), 5, 16)


def check_slots(lens, add, tables, page, n, table_dev=None):
    want = do.slots(lens, add, tables, page, n)
    got = ps.slot_map(to_dev(lens), to_dev(add), to_dev(tables) if table_dev is None else table_dev, page, n)
    for g, w, name in zip(got, want, ("slots", "positions", "requests", "offsets")):
        assert np.array_equal(to_host(g), w), name


@pytest.mark.parametrize("page", [1, 24, 64])
@pytest.mark.parametrize("requests", REQUESTS)
def test_slots(requests, page):
    print(f"slots requests={requests} page={page}", flush=True)
    lens, add, tables, _, _ = make(requests, page, 200, 37, -(-237 // page), 70 + requests)
    total = int(add.sum())
    for n in (0, total // 2, total, total + 501):
        check_slots(lens, add, tables, page, n)
    check_slots(lens, add, tables[:, :2].copy(), page, total + 3)  # columns missing


def test_slots_empty_requests_and_a_long_one():
    """Requests without tokens around one whose tokens fill many turns; a shared table row."""
    lens = np.zeros(5000, dtype=np.int32)
    add = np.zeros(5000, dtype=np.int32)
    add[[0, 4095, 4096, 4999]] = [1, 100_003, 2, 50_000]
    lens[4095] = 77
    row = np.random.default_rng(3).permutation(7000).astype(np.int32)[None, :]
    shared = to_dev(row).expand(5000, 7000)
    check_slots(lens, add, np.broadcast_to(row, (5000, 7000)), 16, 150_010, shared)


def test_slots_far_positions_and_pages():
    """Positions up to 2^31 - 1 and slots past 2^32."""
    top = 2**31 - 1
    for page, columns in ((1 << 20, 2048), ((1 << 24) - 3, 129), (top, 1)):
        lens = np.array([top - 5, 0, top - 1000], dtype=np.int32)
        add = np.array([5, 7, 999], dtype=np.int32)
        tables = (top - np.arange(3 * columns, dtype=np.int64).reshape(3, columns)).astype(np.int32)
        check_slots(lens, add, tables, page, 1011)


def check_release(lens, finished, tables, free, count, page):
    want = do.release(lens, finished, tables, free, count, page)
    f = to_dev(free)
    left = ps.pages_release(to_dev(lens), to_dev(finished), to_dev(tables), f, torch.tensor([count], device=DEV), page)
    assert np.array_equal(to_host(f), want[0])
    assert int(to_host(left)[0]) == want[1]


@pytest.mark.parametrize("share", [0.0, 0.1, 1.0])
@pytest.mark.parametrize("requests", REQUESTS)
def test_release(requests, share):
    print(f"release requests={requests} share={share}", flush=True)
    for page in (1, 16):
        lens, _, tables, free, count = make(requests, page, 12 * page, 0, 13, 90 + requests)
        finished = np.random.default_rng(requests).random(requests) < share
        check_release(lens, finished, tables, free, count, page)
        check_release(lens, finished, tables, free[:len(free) // 2].copy(), count // 3, page)  # the list is too short
        check_release(lens, finished, tables[:, :5].copy(), free, count, page)
    check_release(lens, finished, tables, free, -4, 16)


def test_table_offsets_past_32_bits():
    """Rows of the table that start past 2^32 bytes and past 2^31 elements."""
    stride, columns = (1 << 31) + 5, 40
    wide = torch.empty(stride + columns, dtype=torch.int32, device=DEV)
    t = wide.as_strided((2, columns), (stride, 1))
    tables = np.arange(80, dtype=np.int32).reshape(2, columns)
    t.copy_(to_dev(tables))
    lens, add = np.array([100, 90], dtype=np.int32), np.array([300, 500], dtype=np.int32)
    check_slots(lens, add, tables, 16, 900, t)
    free = np.arange(500, 700, dtype=np.int32)
    want = do.append(lens, add, tables, free, 200, 16)
    ps.pages_append(to_dev(lens), to_dev(add), t, to_dev(free), torch.tensor([200], device=DEV), 16)
    assert np.array_equal(to_host(t), want[0])
    f = to_dev(free)
    ps.pages_release(to_dev(lens), to_dev(np.array([False, True])), t, f, torch.tensor([10], device=DEV), 16)
    assert np.array_equal(to_host(f), do.release(lens, [False, True], want[0], free, 10, 16)[0])


def test_one_page_count_after_the_other():
    """Append, then release: the free list holds every page again, once."""
    lens, add, tables, free, count = make(300, 16, 500, 90, 40, 5)
    total = sorted(np.concatenate([tables[tables >= 0], free[:count]]).tolist())
    t, f = to_dev(tables), to_dev(free)
    left, granted = ps.pages_append(to_dev(lens), to_dev(add), t, f, torch.tensor([count], device=DEV), 16)
    grown = to_dev(lens) + to_dev(add) * granted
    after = ps.pages_release(grown, torch.ones(300, dtype=torch.bool, device=DEV), t, f, left, 16)
    n = int(to_host(after)[0])
    assert sorted(to_host(f)[:n].tolist()) == total


def test_binding_refuses():
    i = torch.zeros(4, dtype=torch.int32, device=DEV)
    t = torch.zeros(4, 8, dtype=torch.int32, device=DEV)
    c = torch.zeros(1, dtype=torch.int64, device=DEV)
    f = torch.zeros(4, dtype=torch.bool, device=DEV)
    out = torch.zeros(1, dtype=torch.int64, device=DEV)
    cases = [
        (TypeError, lambda: ps.pages_append(i.long(), i, t, i, c, 16)),
        (TypeError, lambda: ps.pages_append(i, i, t.long(), i, c, 16)),
        (TypeError, lambda: ps.pages_append(i, i, t, i, c.int(), 16)),
        (ValueError, lambda: ps.pages_append(i[:3], i, t, i, c, 16)),
        (ValueError, lambda: ps.pages_append(i, i, t.t(), i, c, 16)),
        (ValueError, lambda: ps.pages_append(i, i, t[:1].expand(4, 8), i, c, 16)),
        (ValueError, lambda: ps.pages_append(i, i, t, i, c, 0)),
        (ValueError, lambda: ps.pages_append(i, i.cpu(), t, i, c, 16)),
        (ps.LibscanError, lambda: ps.pages_append(i, i, t, t.view(-1), c, 16)),
        (ps.LibscanError, lambda: ps.pages_append(i, i, t, i, c, 16, count_out=c)),
        (ps.LibscanError, lambda: ps.pages_release(i, f, t, i.clone(), c, 16, count_out=c)),
        (ps.LibscanError, lambda: ps.pages_release(i, f, t, i, c, 16)),
        (TypeError, lambda: ps.pages_release(i, i, t, i.clone(), c, 16)),
        (ValueError, lambda: ps.slot_map(i, i, t, 16, -1)),
        (ValueError, lambda: ps.slot_map(i, i, t, 1 << 31, 4)),
        (ValueError, lambda: ps.slot_map(i, i, t.view(-1), 16, 4)),
    ]
    for kind, call in cases:
        with pytest.raises(kind):
            call()
    ps.pages_append(i, i, t, torch.zeros(9, dtype=torch.int32, device=DEV), c, 16, count_out=out)


def test_graph_replays():
    lens, add, tables, free, count = make(500, 16, 400, 60, 40, 8)
    finished = np.random.default_rng(1).random(500) < 0.3
    n = int(add.sum()) + 40
    dl, da, dt, df = to_dev(lens), to_dev(add), to_dev(tables), to_dev(free)
    dc, dfin = torch.tensor([count], device=DEV), to_dev(finished)
    left, granted = torch.empty(1, dtype=torch.int64, device=DEV), torch.empty(500, dtype=torch.bool, device=DEV)
    back = torch.empty(1, dtype=torch.int64, device=DEV)
    out = ps.slot_map(dl, da, dt, 16, n)

    def work():
        ps.pages_append(dl, da, dt, df, dc, 16, left, granted)
        ps.slot_map(dl, da, dt, 16, n, out)
        ps.pages_release(dl, dfin, dt, df, left, 16, back)

    want_t, want_g, want_left = do.append(lens, add, tables, free, count, 16)
    want_s = do.slots(lens, add, want_t, 16, n)
    want_f, want_back = do.release(lens, finished, want_t, free, want_left, 16)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work()
    for rep in range(4):
        dt.copy_(to_dev(tables))
        df.copy_(to_dev(free))
        for o in (*out, left, back, granted):
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(to_host(dt), want_t), rep
        assert np.array_equal(to_host(granted), want_g), rep
        assert int(left) == want_left and int(back) == want_back, rep
        assert np.array_equal(to_host(df), want_f), rep
        for a, b in zip(out, want_s):
            assert np.array_equal(to_host(a), b), rep
        ps.slot_map(dl, da, dt, 16, 7)
        torch.cuda.synchronize()
