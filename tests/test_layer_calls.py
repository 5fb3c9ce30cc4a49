"""The layer's calls on the CPU: what is answered before anything is allocated or enqueued."""
import pytest
import torch

import prefix_scan_stream_amd as ps
from test_layer_abi import A, BACK, RECUR, lib, status  # noqa: F401  (lib is a fixture)


@pytest.mark.parametrize("offsets", [None, A[9]])
@pytest.mark.parametrize("ws", [dict(ws=None, ws_bytes=0), dict(ws_bytes=256)], ids=str)
def test_too_many_tiles_are_refused_before_the_workspace(lib, offsets, ws):  # noqa: F811
    """2^31 - 1 tokens of a channel are 2^24 tiles: a caller is told so, and not to come back with gigabytes."""
    many = dict(sequences=1, rows=(1 << 31) - 1, channels=1, x_s=0, x_r=0, g_s=0, g_r=0, offsets=offsets, **ws)
    assert status(lib, "gated_recurrence", RECUR, **many, o_s=0, o_r=1) == ps.LS_ERR_UNSUPPORTED
    assert status(lib, "gated_recurrence_backward", BACK, **many, do_s=0, do_r=0, dx=A[10], dx_s=0, dx_r=1, dg=A[11], dg_s=0,
                  dg_r=1) == ps.LS_ERR_UNSUPPORTED
    # what is wrong with the arguments comes first
    assert status(lib, "gated_recurrence", RECUR, **many, o_s=0, o_r=0) == ps.LS_ERR_INVALID_ARG
    # a quarter of the rows fit, and want their workspace
    many["rows"] >>= 2
    assert status(lib, "gated_recurrence", RECUR, **many, o_s=0, o_r=1) == ps.LS_ERR_WORKSPACE


@pytest.mark.parametrize("kind", ["recurrence", "experts"])
@pytest.mark.parametrize("capturing", [False, True])
@pytest.mark.parametrize("held", [False, True])
def test_a_refused_call_makes_no_workspace(monkeypatch, kind, capturing, held):
    made = []
    monkeypatch.setattr(ps, "_raw_stream", lambda index: 7)
    monkeypatch.setattr(ps, "_capture_of", lambda handle: 3 if capturing else None)
    monkeypatch.setattr(ps, "_ws_cache", {(0, 7, kind): torch.zeros(64, dtype=torch.uint8)} if held else {})
    monkeypatch.setattr(ps, "workspace_for", lambda *a: made.append(a))
    need = lambda: made.append("size")
    for refusal in (ps.LS_ERR_INVALID_ARG, ps.LS_ERR_UNSUPPORTED):
        st, _ = ps._with_workspace(lambda *a: refusal, (1, 2), kind, 0, need)
        assert st == refusal and made == []


@pytest.fixture
def allocations(monkeypatch):
    """Which way outputs are made: the quick one, or torch's own call, on the CPU."""
    made, strided = [], torch.empty_strided

    def quick(shape, stride, dtype):
        made.append("quick")
        return strided(shape, stride, dtype=dtype)

    def own(shape, stride, *, dtype, device):
        made.append("torch")
        assert device == "cuda"
        return strided(shape, stride, dtype=dtype)

    monkeypatch.setattr(ps, "_quick_empty", quick)
    monkeypatch.setattr(ps, "_quick_empty_holds", None)
    monkeypatch.setattr(ps, "_is_as_asked", lambda t, *asked: (t.dtype, tuple(t.shape), t.stride()) == (asked[2], *asked[:2]))
    monkeypatch.setattr(torch, "empty_strided", own)
    return made


def outputs():
    return ps._vector_of(5, torch.int64), ps._matrix_of(3, 4, torch.float16), ps._rows_of((2, 3, 4), torch.float32)


def test_outputs_are_made_the_quick_way(allocations):
    for t, shape in zip(outputs(), ((5,), (3, 4), (2, 3, 4))):
        assert t.shape == shape and t.is_contiguous()
    assert "torch" not in allocations


def test_outputs_follow_torch_where_it_fills_or_watches(allocations):
    """Deterministic mode fills new tensors, and a dispatch mode sees them: neither is gone round."""
    from torch.utils._python_dispatch import TorchDispatchMode

    class Mode(TorchDispatchMode):
        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            return func(*args, **(kwargs or {}))

    outputs()
    del allocations[:]
    torch.use_deterministic_algorithms(True)
    try:
        outputs()
    finally:
        torch.use_deterministic_algorithms(False)
    assert allocations == ["torch"] * 3
    with Mode():
        outputs()
    assert allocations == ["torch"] * 6
    outputs()
    assert allocations == ["torch"] * 6 + ["quick"] * 3


@pytest.mark.parametrize("changed", ["signature", "type", "order", "missing"])
def test_outputs_without_the_quick_way(monkeypatch, allocations, changed):
    """A torch build whose inner function is not there or not the same: torch's own call serves."""
    strided = torch._C._VariableFunctions.empty_strided

    def other(a, b, c):
        if changed == "signature":
            raise TypeError("_empty_strided_cuda(): incompatible arguments")
        return strided(a, b, dtype=torch.float64) if changed == "type" else strided(a, tuple(reversed(b)), dtype=c)

    monkeypatch.setattr(ps, "_quick_empty", None if changed == "missing" else other)
    for t, (shape, dtype) in zip(outputs(), (((5,), torch.int64), ((3, 4), torch.float16), ((2, 3, 4), torch.float32))):
        assert t.shape == shape and t.dtype is dtype and t.is_contiguous()
    assert allocations == ["torch"] * 3
