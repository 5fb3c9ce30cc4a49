"""The binding's workspaces, on the CPU: which buffer a call gets and which fills are
enqueued for it, with host memory in place of the device's and streams and captures made up."""
import gc
import threading
import time
import weakref
from contextlib import nullcontext
from types import SimpleNamespace

import pytest
import torch

import prefix_scan_stream_amd as ps

CPU = torch.device("cpu")


@pytest.fixture
def fills(monkeypatch):
    """Captures by stream handle, and the (buffer's address, capture) of each fill."""
    state = SimpleNamespace(capture={}, log=[], made=getattr(ps, "_new_workspace", None))

    def init(ws, stream):
        ws.zero_()
        state.log.append((ws.data_ptr(), state.capture.get(stream.cuda_stream)))

    def new(device, stream, nbytes, fill=None):
        ws = torch.empty((max(nbytes, 1 << 16) + 255) & ~255, dtype=torch.uint8)
        init(ws[:fill], stream)
        return ws

    monkeypatch.setattr(ps, "ls_workspace_init", init)
    monkeypatch.setattr(ps, "_new_workspace", new, raising=False)
    monkeypatch.setattr(ps, "_capture_of", lambda handle: state.capture.get(handle), raising=False)
    for name in ("_ws_cache", "_ws_graph", "_ws_uses"):
        monkeypatch.setattr(ps, name, {}, raising=False)
    monkeypatch.setattr(ps, "_ws_retired", [])
    return state


def stream(handle):
    return SimpleNamespace(cuda_stream=handle)


def alive(ws):
    return any(ws is held for held in [*ps._ws_cache.values(), *(kept for _, kept in ps._ws_retired)])


KINDS = ["status", "sort", "phases", "sample"]


@pytest.mark.parametrize("kind", KINDS)
def test_a_graph_counts_on_its_own_fill_only(fills, kind):
    """Two captures on a stream without a workspace, the second no larger: each has a buffer
    and a fill of its own, and an eager call there counts on neither."""
    s = stream(7)
    fills.capture[7] = 1
    a = ps.workspace_for(CPU, s, 100_000, kind)
    assert ps.workspace_for(CPU, s, 90_000, kind) is a
    assert fills.log == [(a.data_ptr(), 1)]
    fills.capture[7] = 2
    b = ps.workspace_for(CPU, s, 90_000, kind)
    assert b is not a and fills.log[1:] == [(b.data_ptr(), 2)]
    bigger = ps.workspace_for(CPU, s, 300_000, kind)
    assert bigger.numel() >= 300_000 and fills.log[2:] == [(bigger.data_ptr(), 2)]
    del fills.capture[7]
    c = ps.workspace_for(CPU, s, 90_000, kind)
    assert c is not a and c is not b and c is not bigger and fills.log[3:] == [(c.data_ptr(), None)]


@pytest.mark.parametrize("kind", KINDS)
def test_a_graph_takes_the_workspace_of_a_stream_that_was_warmed_up(fills, kind):
    """No fill in the first graph; the buffer is kept for it and nobody else has it again."""
    s = stream(9)
    warm = ps.workspace_for(CPU, s, 100_000, kind)
    fills.capture[9] = 5
    assert ps.workspace_for(CPU, s, 100_000, kind) is warm and len(fills.log) == 1
    assert ps.workspace_for(CPU, s, 50_000, kind) is warm and alive(warm)
    del fills.capture[9]
    eager = ps.workspace_for(CPU, s, 50_000, kind)
    assert eager is not warm and fills.log[1:] == [(eager.data_ptr(), None)]
    assert ps.workspace_for(CPU, s, 50_000, kind) is eager
    fills.capture[9] = 6
    assert ps.workspace_for(CPU, s, 50_000, kind) is eager and alive(warm) and alive(eager)


def test_graphs_take_no_more_than_so_much(fills, monkeypatch):
    """A program that warms up and captures again and again: what is kept for its graphs ends at the
    limit, and graphs past it have their own fill."""
    monkeypatch.setattr(ps, "WORKSPACES_TAKEN_BYTES", 5 << 16)
    s, taken = stream(13), 0
    for capture in range(1, 20):
        warm = ps.workspace_for(CPU, s, 1 << 16)
        fills.capture[13] = capture
        ws = ps.workspace_for(CPU, s, 1 << 16)
        assert ws is warm or fills.log[-1] == (ws.data_ptr(), capture)
        taken += ws is warm
        del fills.capture[13]
    assert taken == 5 == len(ps._ws_retired)


@pytest.mark.parametrize("kind,filled", [("status", 70_144), ("sample", 70_144), ("sort", 256), ("phases", 256)])
def test_fill_of_a_graphs_own_workspace(fills, monkeypatch, kind, filled):
    """Plain scratch is not filled at every replay, its header apart."""
    log = []
    monkeypatch.setattr(ps, "ls_workspace_init", lambda ws, s: log.append(ws.numel()))
    monkeypatch.setattr(ps, "_new_workspace", fills.made)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: nullcontext())
    fills.capture[14] = 1
    assert ps.workspace_for(CPU, stream(14), 70_000, kind).numel() == 70_144 and log == [filled]


def test_error_bits_of_a_graphs_workspace_are_reported(fills, monkeypatch):
    """A call in a graph that gave up a wait shows on the stream it was captured on, whether the
    graph took the stream's workspace or has one of its own."""
    monkeypatch.setattr(ps, "ls_workspace_check", lambda ws, s: int(ws[8]))
    s, device = stream(11), SimpleNamespace(index=None)
    monkeypatch.setattr(torch, "device", lambda d: d)
    assert ps.workspace_error_flags(device, s) == 0
    ps.workspace_for(CPU, s, 1000)
    buffers = []
    for capture in (1, 2, 3):
        fills.capture[11] = capture
        buffers.append(ps.workspace_for(CPU, s, 1000))
    del fills.capture[11]
    buffers.append(ps.workspace_for(CPU, s, 1000))
    assert ps.workspace_error_flags(device, s) == 0
    for bit, ws in ((1, buffers[0]), (2, buffers[2]), (4, buffers[3])):  # taken, the last graph's own, eager
        ws[8] = bit
    assert ps.workspace_error_flags(device, s) == 7
    assert ps.workspace_error_flags(device, stream(12)) == 0


def test_two_streams_of_one_capture(fills):
    """Branches of a graph may run side by side."""
    fills.capture.update({3: 1, 4: 1})
    assert ps.workspace_for(CPU, stream(3), 1000) is not ps.workspace_for(CPU, stream(4), 1000)


def test_the_null_stream_is_never_captured():
    assert ps._capture_of(0) is None


# ------------------------------------------------------------ host threads

class Library:
    """Stands for the library: a call on the workspace has to come from the thread that last
    looked one up, and no other call may be under way."""

    def __init__(self):
        self.owner, self.inside, self.broken, self.calls = None, 0, [], 0

    def lookup(self, *args):
        self.owner = threading.get_ident()
        time.sleep(0.002)
        return torch.empty(1 << 16, dtype=torch.uint8)

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *args: ps.LS_OK

        def call(*args):
            self.inside += 1
            if self.owner != threading.get_ident() or self.inside != 1:
                self.broken.append(name)
            time.sleep(0.002)
            self.inside -= 1
            self.calls += 1
            return ps.LS_OK
        return call


def _entry_points():
    x, f = torch.zeros(32, dtype=torch.int32), torch.zeros(32, dtype=torch.uint8)
    logits, one = torch.zeros(2, 16), torch.ones(2)
    return {
        "scan_inclusive": lambda: ps.scan_inclusive(x), "scan_exclusive": lambda: ps.scan_exclusive(x),
        "scan_ex": lambda: ps.scan_ex(x, scheme="reduce_then_scan"),
        "segmented_scan": lambda: ps.segmented_scan(x, heads=f),
        "segmented_scan_offsets": lambda: ps.segmented_scan(x, offsets=torch.tensor([0, 32])),
        "compact_if": lambda: ps.compact_if(x, "lt", 1), "compact_flags": lambda: ps.compact_flags(x, f),
        "select_indices_if": lambda: ps.select_indices_if(x, "lt", 1),
        "select_indices_flags": lambda: ps.select_indices_flags(f), "radix_sort": lambda: ps.radix_sort(x),
        "sample_tokens": lambda: ps.sample_tokens(logits, one, one, top_p=one),
    }


@pytest.mark.parametrize("name", list(_entry_points()))
def test_a_call_keeps_its_workspace_while_it_enqueues(name, monkeypatch):
    """Two host threads on one stream: from the lookup of the workspace to the end of the
    library's call neither comes between the other's."""
    lib, call = Library(), _entry_points()[name]
    monkeypatch.setattr(ps, "_lib", lib)
    monkeypatch.setattr(ps, "load_library", lambda: lib)
    monkeypatch.setattr(ps, "_require_gpu", lambda *t: None)
    monkeypatch.setattr(ps, "_stream_handle", lambda device: (stream(0), 0))
    monkeypatch.setattr(ps, "_current_device", lambda: -1)
    monkeypatch.setattr(ps, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(ps, "workspace_for", lib.lookup)
    monkeypatch.setattr(ps, "_sample_workspace", lib.lookup)
    monkeypatch.setattr(ps, "_checked", False)
    threads = [threading.Thread(target=lambda: [call() for _ in range(5)]) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert lib.calls == 10 and not lib.broken


# ------------------------------------------------------------ growth

def test_growing_batches_make_few_workspaces_and_keep_one(fills, monkeypatch):
    """A batch that grows by a row a step: the buffers are made a few times, none that was
    replaced is kept, and the last is at most about twice the need."""
    made, new = [], ps._new_workspace
    monkeypatch.setattr(ps, "_new_workspace", lambda *a: made.append(weakref.ref(w := new(*a))) or w, raising=False)
    for rows in range(1, 513):
        need = ps.ls_sample_workspace_bytes(rows, 131072)
        ws = ps.workspace_for(CPU, stream(0), need, "sample")
        assert ws.numel() >= need
    assert len(made) < 16 and ws.numel() <= 2 * need + 256
    gc.collect()
    assert [ref() is not None for ref in made] == [False] * (len(made) - 1) + [True]
    assert not ps._ws_retired


def test_large_workspaces_grow_to_their_need(fills):
    """No doubling where that would take a large part of the memory."""
    limit = ps.WORKSPACE_DOUBLING_BYTES
    ps.workspace_for(CPU, stream(0), limit, "sort")
    assert ps.workspace_for(CPU, stream(0), limit + 5, "sort").numel() < limit + 512
