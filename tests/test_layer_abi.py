"""Refusals of the gated recurrence and the experts' calls, on the CPU: every call here fails its
checks before any GPU work (the addresses are never dereferenced); and the oracle by hand."""
import ctypes

import numpy as np
import pytest
import torch

import layer_oracle as lo
import prefix_scan_stream_amd as ps

INV, WS = ps.LS_ERR_INVALID_ARG, ps.LS_ERR_WORKSPACE
A = [0x7F0000000000 + i * 0x1000000000 for i in range(16)]


@pytest.fixture(scope="module")
def lib():
    return ps.load_library()


# float32, 3 sequences of 500 tokens of 64 channels, x and gate halves of one matrix
RECUR = dict(x=A[0], x_s=64000, x_r=128, g=A[0] + 256, g_s=64000, g_r=128, out=A[1], o_s=32000, o_r=64, state=A[2], st=64,
             state_out=A[3], so=64, carries=A[4], offsets=None, sequences=3, rows=500, channels=64, t=0, gating=2, ws=A[5],
             ws_bytes=1 << 40)
BACK = dict(dout=A[6], do_s=32000, do_r=64, x=A[0], x_s=64000, x_r=128, g=A[0] + 256, g_s=64000, g_r=128, carries=A[4],
            state=A[2], st=64, dstate_out=A[3], dso=64, dx=A[7], dx_s=64000, dx_r=128, dg=A[7] + 256, dg_s=64000, dg_r=128,
            dstate=A[8], ds=64, offsets=None, sequences=3, rows=500, channels=64, t=0, gating=2, ws=A[5], ws_bytes=1 << 40)
SORT = dict(experts=A[0], bits=64, pairs=100, num=8, offsets=A[1], order=A[2], places=A[3], ws=A[4], ws_bytes=1 << 30)
GATHER = dict(x=A[0], xs=64, places=A[1], rows=A[2], rs=64, tokens=10, top=4, num_rows=40, channels=64, t=0)
COMBINE = dict(rows=A[0], rs=64, places=A[1], w=A[2], wt=0, out=A[3], os=64, tokens=10, top=4, num_rows=40, channels=64, t=0)
CBACK = dict(dout=A[0], ds=64, rows=A[1], rs=64, places=A[2], w=A[3], wt=0, drows=A[4], drs=64, dw=A[5], tokens=10, top=4,
             num_rows=40, channels=64, t=0)


def status(lib, name, base, **change):
    return getattr(lib, name)(*{**base, **change}.values(), None)


SIZES = [dict(sequences=-1), dict(sequences=1 << 31), dict(rows=-1), dict(rows=1 << 31), dict(channels=-1),
         dict(channels=(1 << 23) + 1), dict(t=3), dict(t=-1), dict(gating=3), dict(gating=-1), dict(ws=A[5] + 8)]


@pytest.mark.parametrize("change", SIZES + [
    dict(x=None), dict(x=A[0] + 2), dict(g=None), dict(g=A[0] + 1), dict(out=None), dict(out=A[1] + 2), dict(state=A[2] + 2),
    dict(state_out=None), dict(state_out=A[3] + 2), dict(carries=A[4] + 1), dict(x_s=-1), dict(x_r=-128), dict(g_r=-1),
    dict(o_r=63), dict(o_s=-1), dict(o_s=31999), dict(so=63), dict(st=-1), dict(x_s=1 << 62), dict(g_r=1 << 61),
    dict(out=A[0]), dict(out=A[0], o_s=64000, o_r=128), dict(out=A[0] + 128, o_s=64000, o_r=128), dict(out=A[2]),
    dict(state_out=A[2] + 4), dict(state=A[3], st=128), dict(state_out=A[0] + 512), dict(carries=A[1]), dict(carries=A[3]),
    dict(ws=A[1]), dict(ws=A[4]), dict(offsets=A[6] + 4), dict(offsets=A[1]), dict(offsets=A[3], state=None)], ids=str)
def test_recurrence_refuses(lib, change):
    assert status(lib, "gated_recurrence", RECUR, **change) == INV


def test_recurrence_refuses_too_many_tiles(lib):
    """2^31 - 1 tokens of a channel are 2^24 tiles: more than a launch holds."""
    many = dict(sequences=1, rows=(1 << 31) - 1, channels=1, x_s=0, x_r=0, g_s=0, g_r=0)
    for offsets in (None, A[9]):
        assert status(lib, "gated_recurrence", RECUR, **many, o_s=0, o_r=1, offsets=offsets) == ps.LS_ERR_UNSUPPORTED
        assert status(lib, "gated_recurrence_backward", BACK, **many, do_s=0, do_r=0, dx=A[10], dx_s=0, dx_r=1, dg=A[11], dg_s=0,
                      dg_r=1, offsets=offsets) == ps.LS_ERR_UNSUPPORTED


@pytest.mark.parametrize("change", SIZES + [
    dict(dout=None), dict(dout=A[6] + 3), dict(x=None), dict(g=None), dict(carries=None), dict(carries=A[4] + 2),
    dict(state=A[2] + 1), dict(dstate_out=A[3] + 2), dict(dx=None), dict(dg=None), dict(dx=A[7] + 2), dict(dstate=None),
    dict(dx=A[6], dx_s=32000, dx_r=64), dict(dg=A[7]), dict(dg=A[7] + 128), dict(dx=A[0]), dict(dstate=A[2]), dict(dstate=A[3]),
    dict(dx_r=64), dict(dx_r=63), dict(ds=63), dict(dg_s=100), dict(do_s=-1), dict(dso=-1), dict(dx=A[4]), dict(ws=A[8]),
    dict(offsets=A[8])], ids=str)
def test_recurrence_backward_refuses(lib, change):
    assert status(lib, "gated_recurrence_backward", BACK, **change) == INV


@pytest.mark.parametrize("change", [dict(bits=16), dict(bits=0), dict(pairs=-1), dict(pairs=1 << 31), dict(num=0), dict(num=-1),
                                    dict(num=1025), dict(experts=None), dict(experts=A[0] + 4), dict(offsets=None),
                                    dict(offsets=A[1] + 4), dict(order=None), dict(order=A[2] + 2), dict(places=A[3] + 1),
                                    dict(places=A[2]), dict(order=A[0] + 40), dict(offsets=A[3]), dict(ws=A[4] + 4),
                                    dict(ws=A[2]), dict(ws=A[0])], ids=str)
def test_sort_refuses(lib, change):
    assert status(lib, "experts_sort", SORT, **change) == INV


MOVES = [dict(tokens=-1), dict(tokens=1 << 31), dict(top=-1), dict(top=1 << 31), dict(tokens=1 << 20, top=1 << 12),
         dict(num_rows=-1), dict(num_rows=1 << 31), dict(channels=-1), dict(channels=(1 << 23) + 1), dict(t=3), dict(places=None)]


@pytest.mark.parametrize("change", MOVES + [dict(x=None), dict(x=A[0] + 2), dict(xs=-1), dict(rows=None), dict(rows=A[2] + 1),
                                            dict(rs=63), dict(rs=-1), dict(rows=A[0]), dict(rows=A[1]), dict(places=A[1] + 2),
                                            dict(xs=1 << 62), dict(rs=1 << 60)], ids=str)
def test_gather_refuses(lib, change):
    assert status(lib, "experts_gather", GATHER, **change) == INV


@pytest.mark.parametrize("change", MOVES + [dict(rows=None), dict(rows=A[0] + 2), dict(rs=-1), dict(w=A[2] + 2), dict(wt=4),
                                            dict(out=None), dict(out=A[3] + 1), dict(os=63), dict(out=A[0] + 64),
                                            dict(out=A[2]), dict(out=A[1])], ids=str)
def test_combine_refuses(lib, change):
    assert status(lib, "experts_combine", COMBINE, **change) == INV


@pytest.mark.parametrize("change", MOVES + [dict(dout=None), dict(rows=None), dict(w=None), dict(w=A[3] + 1), dict(wt=-1),
                                            dict(drows=None), dict(drs=63), dict(dw=None), dict(dw=A[5] + 2), dict(drows=A[1]),
                                            dict(drows=A[0]), dict(dw=A[3]), dict(dw=A[4] + 64), dict(dw=A[2])], ids=str)
def test_combine_backward_refuses(lib, change):
    assert status(lib, "experts_combine_backward", CBACK, **change) == INV


def test_workspaces(lib):
    size, rows = ctypes.c_size_t(0), ctypes.c_int64(0)
    need = ctypes.byref(size)
    assert lib.ls_experts_workspace_bytes(1 << 20, 256, need) == ps.LS_OK and size.value >= 256
    assert status(lib, "experts_sort", SORT, ws=None) == WS and status(lib, "experts_sort", SORT, ws_bytes=8) == WS
    for pairs, num, out in ((-1, 8, need), (1 << 31, 8, need), (8, 0, need), (8, 1025, need), (8, 8, None)):
        assert lib.ls_experts_workspace_bytes(pairs, num, out) == INV
    good = (3, 500, 64, 0, 0)
    assert lib.ls_recurrence_workspace_bytes(*good, need) == ps.LS_OK
    if size.value > 0:
        assert status(lib, "gated_recurrence", RECUR, ws=None) == WS
        assert status(lib, "gated_recurrence", RECUR, ws_bytes=size.value - 1) == WS
    for i, v in ((0, -1), (0, 1 << 31), (1, -1), (1, 1 << 31), (2, -1), (2, (1 << 23) + 1), (4, 3)):
        bad = list(good)
        bad[i] = v
        assert lib.ls_recurrence_workspace_bytes(*bad, need) == INV
    assert lib.ls_recurrence_workspace_bytes(*good, None) == INV
    assert lib.ls_recurrence_carry_rows(3, 500, 0, ctypes.byref(rows)) == ps.LS_OK and rows.value == 3 * 8
    assert lib.ls_recurrence_carry_rows(3, 500, 1, ctypes.byref(rows)) == ps.LS_OK and rows.value == 8
    assert lib.ls_recurrence_carry_rows(-1, 500, 1, ctypes.byref(rows)) == INV
    assert lib.ls_recurrence_carry_rows(3, 500, 1, None) == INV


def test_binding_refuses_cpu_tensors():
    x, p = torch.zeros(2, 5, 8), torch.zeros(2, 1, dtype=torch.int32)
    for call in (lambda: ps.gated_recurrence(x, x), lambda: ps.gated_recurrence_backward(x, x, x, x),
                 lambda: ps.recurrence_carries(x), lambda: ps.experts_sort(p, 4), lambda: ps.experts_gather(x[0], p),
                 lambda: ps.experts_combine(x[0], p), lambda: ps.experts_combine_backward(x[0], x[0], p, p.float())):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------ the oracle on worked examples

def test_oracle_recurrence_by_hand():
    x, g = np.array([[[1.0], [2.0], [3.0]]]), np.array([[[0.5], [0.5], [2.0]]])
    h, _, last = lo.recurrence(x, g, np.array([[4.0]]), "decay")
    assert h.ravel().tolist() == [3.0, 3.5, 10.0] and last.tolist() == [[10.0]]
    h, _, _ = lo.recurrence(x, np.zeros_like(g), None, "sigmoid")  # a = 1/2
    assert h.ravel().tolist() == [0.5, 1.25, 2.125]
    h, _, _ = lo.recurrence(x, np.log(g), np.array([[4.0]]), "log")
    assert np.allclose(h.ravel(), [3.0, 3.5, 10.0], rtol=1e-15)
    (dx, dg, ds), _ = lo.gradients(x, g, np.array([[4.0]]), np.ones_like(x), None, "decay")
    # lambda from behind: 1, 1 + 2 * 1, 1 + 0.5 * 3
    assert dx.ravel().tolist() == [2.5, 3.0, 1.0] and dg.ravel().tolist() == [10.0, 9.0, 3.5] and ds.tolist() == [[1.25]]


@pytest.mark.parametrize("gating", ["decay", "log", "sigmoid"])
def test_oracle_gradients_against_differences(gating):
    r = np.random.default_rng(5)
    v = [r.standard_normal((2, 6, 3)), -np.abs(r.standard_normal((2, 6, 3))), r.standard_normal((2, 3))]
    p, q = r.standard_normal((2, 6, 3)), r.standard_normal((2, 3))

    def loss(x, g, s):
        h, _, last = lo.recurrence(x, g, s, gating)
        return (h * p).sum() + (last * q).sum()

    got, _ = lo.gradients(*v, p, q, gating)
    for k in range(3):
        for at in np.ndindex(*v[k].shape):
            e = np.zeros_like(v[k])
            e[at] = 1e-6
            up, down = [a + e if i == k else a for i, a in enumerate(v)], [a - e if i == k else a for i, a in enumerate(v)]
            # the difference's own error: e^2 of the third derivative, and 2^-53 |L| / e
            assert abs((loss(*up) - loss(*down)) / 2e-6 - got[k][at]) < 1e-7


def test_oracle_experts_by_hand():
    e = np.array([[2, 0], [0, -1], [2, 2]])
    offsets, order, places = lo.sort(e, 3)
    assert offsets.tolist() == [0, 2, 2, 5] and order.tolist() == [1, 2, 0, 4, 5, -1]
    assert places.tolist() == [[2, 0], [1, -1], [3, 4]]
    x = np.arange(6.0).reshape(3, 2)
    rows = lo.gather(x, places, np.full((6, 2), 9.0))
    assert rows.tolist() == [[0, 1], [2, 3], [0, 1], [4, 5], [4, 5], [9, 9]]
    w = np.array([[1.0, 2.0], [3.0, 0.0], [0.5, 0.5]])
    assert lo.combine(rows, places, w)[0].tolist() == [[0, 3], [6, 9], [4, 5]]
    drows, dw, _ = lo.combine_backward(x, rows, places, w, np.zeros((6, 2)))
    assert dw.tolist() == [[1, 1], [13, 0], [41, 41]] and drows[1].tolist() == [6, 9] and drows[5].tolist() == [0, 0]
