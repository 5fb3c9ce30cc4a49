"""Refusals of the decoding-step operators, on the CPU: every call here fails its checks
before any GPU work (the addresses are never dereferenced)."""
import ctypes

import numpy as np
import pytest
import torch

import decode_oracle as do
import prefix_scan_stream_amd as ps

INV, WS = ps.LS_ERR_INVALID_ARG, ps.LS_ERR_WORKSPACE
A = [0x7F0000000000 + i * 0x1000000000 for i in range(12)]


@pytest.fixture(scope="module")
def lib():
    return ps.load_library()


SAMPLE = dict(logits=A[0], rows=4, vocab=100, stride=128, t=2, u=A[1], temp=A[2], k=A[3], p=A[4], m=A[5], tokens=A[6],
              logprobs=A[7], ws=A[8], ws_bytes=1 << 30)
APPEND = dict(lens=A[0], new=A[1], requests=4, tables=A[2], columns=10, stride=12, free=A[3], capacity=50, count=A[4],
              page=16, count_out=A[5], granted=A[6])
SLOTS = dict(lens=A[0], new=A[1], requests=4, tables=A[2], columns=10, stride=12, page=16, n=30, slots=A[3],
             positions=A[4], ids=A[5], offsets=A[6])
RELEASE = dict(lens=A[0], finished=A[1], requests=4, tables=A[2], columns=10, stride=12, free=A[3], capacity=50,
               count=A[4], page=16, count_out=A[5])


def status(lib, name, base, **change):
    return getattr(lib, name)(*{**base, **change}.values(), None)


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(vocab=-1), dict(rows=1 << 31), dict(vocab=1 << 31), dict(stride=99), dict(stride=-128),
    dict(t=3), dict(t=-1), dict(logits=None), dict(logits=A[0] + 1), dict(t=0, logits=A[0] + 2), dict(u=None),
    dict(u=A[1] + 2), dict(temp=None), dict(temp=A[2] + 1), dict(k=A[3] + 2), dict(p=A[4] + 1), dict(m=A[5] + 3),
    dict(tokens=None), dict(tokens=A[6] + 4), dict(logprobs=A[7] + 2), dict(ws=A[8] + 8),
    dict(tokens=A[0] + 512), dict(logprobs=A[1] + 8), dict(tokens=A[7]), dict(ws=A[0]), dict(ws=A[6]),
    dict(k=A[6] + 8), dict(m=A[7] + 12),
], ids=str)
def test_sample_refuses(lib, change):
    assert status(lib, "sample_tokens", SAMPLE, **change) == INV


def test_sample_workspace(lib):
    assert status(lib, "sample_tokens", SAMPLE, ws=None) == WS
    assert status(lib, "sample_tokens", SAMPLE, ws_bytes=16) == WS
    size = ctypes.c_size_t(0)
    assert lib.ls_sample_workspace_bytes(4, 100, ctypes.byref(size)) == ps.LS_OK and size.value >= 256
    for rows, vocab, out in ((-1, 5, ctypes.byref(size)), (5, -1, ctypes.byref(size)),
                             (1 << 31, 5, ctypes.byref(size)), (5, 1 << 31, ctypes.byref(size)), (5, 5, None)):
        assert lib.ls_sample_workspace_bytes(rows, vocab, out) == INV
    with pytest.raises(ps.LibscanError):
        ps.ls_sample_workspace_bytes(-1, 5)


def test_strides_past_the_address_range(lib):
    """(rows - 1) * stride elements must not wrap round to a small matrix."""
    for rows, stride in ((1 << 30, 1 << 40), ((1 << 24) + 1, 1 << 40), (3, 1 << 62), (2, (1 << 63) - 1)):
        assert status(lib, "sample_tokens", SAMPLE, rows=rows, stride=stride) == INV
        assert status(lib, "slot_map", SLOTS, requests=rows, stride=stride) == INV
        assert status(lib, "pages_append", APPEND, requests=rows, stride=stride) == INV
        assert status(lib, "pages_release", RELEASE, requests=rows, stride=stride) == INV


COMMON = [dict(requests=-1), dict(requests=1 << 31), dict(columns=-1), dict(columns=1 << 31), dict(stride=9),
          dict(stride=-1), dict(page=0), dict(page=-16), dict(page=1 << 31), dict(lens=None), dict(lens=A[0] + 2),
          dict(tables=None), dict(tables=A[2] + 2)]
LIST = [dict(capacity=-1), dict(free=None), dict(free=A[3] + 1), dict(count=None), dict(count=A[4] + 4),
        dict(count_out=None), dict(count_out=A[5] + 4), dict(count_out=A[4]), dict(count_out=A[3] + 16),
        dict(count_out=A[2] + 48), dict(count_out=A[0])]


@pytest.mark.parametrize("change", COMMON + LIST + [
    dict(new=None), dict(new=A[1] + 1), dict(granted=None), dict(granted=A[0] + 3), dict(granted=A[2] + 100),
    dict(granted=A[5]), dict(tables=A[0]), dict(tables=A[3] + 40), dict(tables=A[4] - 8), dict(stride=0)], ids=str)
def test_append_refuses(lib, change):
    assert status(lib, "pages_append", APPEND, **change) == INV


@pytest.mark.parametrize("change", COMMON + [
    dict(n=-1), dict(new=None), dict(new=A[1] + 3), dict(slots=None), dict(slots=A[3] + 4), dict(positions=None),
    dict(positions=A[4] + 2), dict(ids=None), dict(ids=A[5] + 1), dict(offsets=None), dict(offsets=A[6] + 4),
    dict(slots=A[0]), dict(positions=A[3] + 100), dict(ids=A[2]), dict(offsets=A[1]), dict(offsets=A[4])], ids=str)
def test_slot_map_refuses(lib, change):
    assert status(lib, "slot_map", SLOTS, **change) == INV


@pytest.mark.parametrize("change", COMMON + LIST + [
    dict(finished=None), dict(free=A[2]), dict(free=A[0]), dict(free=A[1])], ids=str)
def test_release_refuses(lib, change):
    assert status(lib, "pages_release", RELEASE, **change) == INV


def test_binding_refuses_cpu_tensors():
    x, f = torch.zeros(2, 5), torch.zeros(2)
    i, t = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 5, dtype=torch.int32)
    c = torch.zeros(1, dtype=torch.int64)
    with pytest.raises(ValueError):
        ps.sample_tokens(x, f, f)
    with pytest.raises(ValueError):
        ps.pages_append(i, i, t, i, c, 16)
    with pytest.raises(ValueError):
        ps.slot_map(i, i, t, 16, 4)
    with pytest.raises(ValueError):
        ps.pages_release(i, i.bool(), t, i, c, 16)


# ------------------------------------------------------------ the oracle on worked examples

def test_oracle_sample_by_hand():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    assert [do.sample_row(x, u, 1.0)[0] for u in (0.0, 0.05, 0.2, 0.55, 0.65, 0.75, 0.99)] == [0, 0, 1, 2, 2, 3, 3]
    # two largest: 0.4 and 0.3
    assert [do.sample_row(x, u, 1.0, top_k=2)[0] for u in (0.0, 0.5, 0.6, 0.99)] == [1, 1, 3, 3]
    assert do.sample_row(x, 0.9, 1.0, top_k=2)[1] == pytest.approx(np.log(3 / 7), rel=1e-14)
    # 0.4 + 0.3 reach 0.65; 0.4 alone reaches 0.39
    assert [do.sample_row(x, u, 1.0, top_p=0.65)[0] for u in (0.0, 0.5, 0.6, 0.99)] == [1, 1, 3, 3]
    assert do.sample_row(x, 0.99, 1.0, top_p=0.39)[0] == 1
    assert [do.sample_row(x, u, 1.0, min_p=0.45)[0] for u in (0.0, 0.45, 0.99)] == [1, 2, 3]
    assert do.sample_row([1.0, 3.0, 3.0], 0.9, 0.0)[:2] == (1, 0.0)
    assert do.sample_row([1.0, 3.0, 3.0], 0.9, 1.0, top_k=1)[0] == 1  # of equal ones the first
    assert do.sample_row([-np.inf, np.nan], 0.5, 1.0)[:2] == (-1, -np.inf)


def test_oracle_cache_by_hand():
    tables = np.array([[7, -1, -1], [8, 9, -1], [5, -1, -1]], dtype=np.int32)
    free = np.array([1, 2, 3, 4], dtype=np.int32)
    t, granted, count = do.append([4, 5, 1], [5, 3, 1], tables, free, 4, 4)
    assert t.tolist() == [[7, 4, 3], [8, 9, -1], [5, -1, -1]] and granted.all() and count == 2
    t, granted, count = do.append([4, 5, 1], [5, 4, 1], tables, free, 1, 4)
    assert granted.tolist() == [False, False, True] and count == 1
    s, p, r, o = do.slots([3, 0], [3, 1], tables, 4, 6)
    assert s.tolist() == [31, -1, -1, 32, -1, -1] and p.tolist() == [3, 4, 5, 0, 0, 0]
    assert r.tolist() == [0, 0, 0, 1, -1, -1] and o.tolist() == [0, 3, 4]
    f, count = do.release([4, 5, 1], [True, True, False], tables, free, 2, 4)
    assert f.tolist() == [1, 2, 7, 8] and count == 5
