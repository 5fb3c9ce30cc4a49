"""prefix_scan_stream_amd -- Python binding of libscan (MI355X / gfx950).

A thin ctypes layer over the C ABI in include/libscan.h: it checks that tensors
live on a GPU, passes their pointers, sizes and the current HIP stream, and
raises LibscanError on a non-OK status.  Every step of the computation runs in
the library's HIP kernels; there is no other implementation behind these names,
and importing or calling them fails loudly when libscan.so is missing.

PyTorch supplies device memory and streams only.  Workspaces are cached per
(device, stream), zero-filled by the library once when they are made, and grown
on demand.  A call that is being captured into a HIP graph uses a workspace of
that graph's own: the stream's cached one, if eager calls have made one, which then
is the graph's and is kept (release_workspaces() frees it); else one from the graph's
memory pool, whose zero fill is part of the graph.  So graphs may be replayed in any
order, between eager calls and on several streams.

Checked mode (set_checked(True), or LIBSCAN_CHECKED=1 in the environment) reads
the workspace's error word after every call that uses one -- which waits for the
stream -- and raises LibscanError(LS_ERR_INCOMPLETE) when a bounded wait inside
the call gave up, re-initialising the workspace.  It is off by default so that
calls stay asynchronous and can be captured in graphs.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np
import torch

__all__ = [
    "LibscanError", "library_path", "load_library", "ls_abi_version", "ls_status_string",
    "ls_scan_workspace_bytes", "ls_compact_workspace_bytes", "scan_inclusive", "scan_exclusive",
    "compact_if", "batched_row_scan", "workspace_for", "scan_ex", "ls_scan_ex_workspace_bytes",
    "batched_row_scan_ex", "radix_sort", "ls_radix_sort_workspace_bytes", "compact_flags",
    "select_indices_if", "select_indices_flags",
    "segmented_scan", "ls_segmented_workspace_bytes", "scan_noalloc", "SCAN_NOALLOC_MAX_N",
    "ls_workspace_init", "ls_workspace_check", "set_checked", "workspace_error_flags",
    "release_workspaces", "sample_tokens", "ls_sample_workspace_bytes", "pages_append", "slot_map",
    "pages_release",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libscan.so")

LS_OK, LS_ERR_INVALID_ARG, LS_ERR_UNSUPPORTED, LS_ERR_WORKSPACE, LS_ERR_HIP, LS_ERR_INCOMPLETE = range(6)
DTYPE_CODES = {"int32": 0, "uint32": 1, "float32": 2}
OP_CODES = {"sum": 0, "max": 1, "xor": 2, "min": 3, "and": 4, "or": 5, "prod": 6, "affine": 7}
CMP_CODES = {"lt": 0, "le": 1, "gt": 2, "ge": 3, "eq": 4, "ne": 5}
SCHEME_CODES = {"single_pass": 0, "reduce_then_scan": 1, "scan_then_propagate": 2,
                "deterministic": 3}
LOGITS_CODES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
BLOCK_SCAN_CODES = {"wave_dpp": 0, "hillis_steele": 1, "hillis_steele_double": 2, "blelloch": 3}
_TORCH_DTYPES = {torch.int32: "int32", torch.float32: "float32"}
if hasattr(torch, "uint32"):
    _TORCH_DTYPES[torch.uint32] = "uint32"

SCAN_NOALLOC_MAX_N = 402653184  # LS_SCAN_NOALLOC_MAX_N

_lock = threading.Lock()
_lib = None
ABI_VERSION = 5  # the libscan.h version this binding marshals for
_checked = os.environ.get("LIBSCAN_CHECKED", "0") not in ("", "0")


class LibscanError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = ls_status_string(status) if _lib is not None else f"status {status}"
        super().__init__(f"{where}: {msg}")


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libscan.so (built in-tree by prefix_scan_stream_amd.build)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise ImportError(
                f"libscan.so not found at {_LIB_PATH}; build it with "
                "`python -m prefix_scan_stream_amd.build`")
        lib = ctypes.CDLL(_LIB_PATH)
        P, I64, I, U32, SZ = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint32,
                              ctypes.c_size_t)
        lib.ls_abi_version.argtypes = []
        lib.ls_abi_version.restype = I
        if lib.ls_abi_version() != ABI_VERSION:
            raise ImportError(f"{_LIB_PATH} has ABI version {lib.ls_abi_version()}, this binding "
                              f"needs {ABI_VERSION}; rebuild with `python -m prefix_scan_stream_amd.build`")
        lib.ls_status_string.argtypes = [I]
        lib.ls_status_string.restype = ctypes.c_char_p
        lib.ls_workspace_init.argtypes = [P, SZ, P]
        lib.ls_workspace_init.restype = I
        lib.ls_workspace_check.argtypes = [P, ctypes.POINTER(U32), P]
        lib.ls_workspace_check.restype = I
        lib.ls_scan_workspace_bytes.argtypes = [I64, I, I, ctypes.POINTER(SZ)]
        lib.ls_scan_workspace_bytes.restype = I
        lib.ls_compact_workspace_bytes.argtypes = [I64, I, ctypes.POINTER(SZ)]
        lib.ls_compact_workspace_bytes.restype = I
        for name in ("scan_inclusive", "scan_exclusive"):
            fn = getattr(lib, name)
            fn.argtypes = [P, P, I64, I, I, P, P, SZ, P]
            fn.restype = I
        lib.ls_scan_ex_workspace_bytes.argtypes = [I64, I, I, I, ctypes.POINTER(SZ)]
        lib.ls_scan_ex_workspace_bytes.restype = I
        lib.scan_ex.argtypes = [P, P, I64, I, I, I, I, P, P, SZ, P]
        lib.ls_segmented_workspace_bytes.argtypes = [I64, I, I, ctypes.POINTER(SZ)]
        lib.ls_segmented_workspace_bytes.restype = I
        lib.segmented_scan.argtypes = [P, P, I64, I, I, I, P, P, P, SZ, P]
        lib.segmented_scan.restype = I
        lib.segmented_scan_offsets.argtypes = [P, P, I64, I, I, I, P, I64, P, P, SZ, P]
        lib.segmented_scan_offsets.restype = I
        lib.scan_ex.restype = I
        lib.batched_row_scan_ex.argtypes = [P, P, I64, I64, I, I, I, I, P]
        lib.batched_row_scan_ex.restype = I
        lib.compact_flags.argtypes = [P, P, P, P, I64, P, SZ, P]
        lib.compact_flags.restype = I
        lib.select_indices_if.argtypes = [P, P, P, I64, I, I, U32, P, SZ, P]
        lib.select_indices_if.restype = I
        lib.select_indices_flags.argtypes = [P, P, P, I64, P, SZ, P]
        lib.select_indices_flags.restype = I
        lib.ls_radix_sort_workspace_bytes.argtypes = [I64, I, I, ctypes.POINTER(SZ)]
        lib.ls_radix_sort_workspace_bytes.restype = I
        lib.radix_sort.argtypes = [P, P, P, P, I64, I, P, SZ, P]
        lib.radix_sort.restype = I
        lib.scan_noalloc.argtypes = [P, P, I64, I, I, I, P, P]
        lib.scan_noalloc.restype = I
        lib.compact_if.argtypes = [P, P, P, I64, I, I, U32, P, SZ, P]
        lib.compact_if.restype = I
        lib.batched_row_scan.argtypes = [P, P, I64, I64, I, I, I, P]
        lib.batched_row_scan.restype = I
        lib.ls_sample_workspace_bytes.argtypes = [I64, I64, ctypes.POINTER(SZ)]
        lib.ls_sample_workspace_bytes.restype = I
        lib.sample_tokens.argtypes = [P, I64, I64, I64, I, P, P, P, P, P, P, P, P, SZ, P]
        lib.sample_tokens.restype = I
        lib.pages_append.argtypes = [P, P, I64, P, I64, I64, P, I64, P, I64, P, P, P]
        lib.pages_append.restype = I
        lib.slot_map.argtypes = [P, P, I64, P, I64, I64, I64, I64, P, P, P, P, P]
        lib.slot_map.restype = I
        lib.pages_release.argtypes = [P, P, I64, P, I64, I64, P, I64, P, I64, P, P]
        lib.pages_release.restype = I
        # of the HIP runtime that libscan.so is linked with
        lib.hipStreamGetCaptureInfo.argtypes = [P, ctypes.POINTER(I), ctypes.POINTER(ctypes.c_ulonglong)]
        lib.hipStreamGetCaptureInfo.restype = I
        _lib = lib
        return lib


def ls_abi_version() -> int:
    return load_library().ls_abi_version()


def ls_status_string(status: int) -> str:
    return load_library().ls_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != LS_OK:
        raise LibscanError(status, where)


def ls_scan_workspace_bytes(n: int, dtype: str, op: str) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().ls_scan_workspace_bytes(n, DTYPE_CODES[dtype], OP_CODES[op],
                                                  ctypes.byref(out)), "ls_scan_workspace_bytes")
    return out.value


def ls_scan_ex_workspace_bytes(n: int, dtype: str, op: str, scheme: str) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().ls_scan_ex_workspace_bytes(n, DTYPE_CODES[dtype], OP_CODES[op],
                                                     SCHEME_CODES[scheme], ctypes.byref(out)),
           "ls_scan_ex_workspace_bytes")
    return out.value


def ls_compact_workspace_bytes(n: int, dtype: str) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().ls_compact_workspace_bytes(n, DTYPE_CODES[dtype], ctypes.byref(out)),
           "ls_compact_workspace_bytes")
    return out.value


# ------------------------------------------------------------ workspaces

# Held from the lookup of a workspace to the end of the call that enqueues on it: the kernels of
# one call stand together on the stream, also where several host threads use that.
_ws_lock = threading.RLock()
_ws_cache: dict = {}    # (device index, stream handle) -> the uint8 workspace in use
_ws_uses: dict = {}     # calls on each cached status workspace since its last initialisation
STATUS_REINIT_CALLS = 1 << 25
_ws_graph: dict = {}    # the same key -> (capture, workspace) of the last graph captured there
_ws_retired: list = []  # (the same key, workspace given to a graph)
WORKSPACE_DOUBLING_BYTES = 64 << 20
WORKSPACES_TAKEN_BYTES = 256 << 20  # most that graphs take of streams' workspaces, as these are kept for good


def set_checked(on: bool = True) -> None:
    """Checked mode: after each call that uses a workspace, wait for the stream and
    raise LibscanError(LS_ERR_INCOMPLETE) if a bounded wait in the call gave up."""
    global _checked
    _checked = bool(on)


def ls_workspace_init(ws: torch.Tensor, stream=None) -> None:
    """Zero-fill a uint8 device workspace (before first use) on `stream` (default:
    the current stream)."""
    _require_gpu(ws)
    s = stream if stream is not None else torch.cuda.current_stream(ws.device)
    _check(load_library().ls_workspace_init(_ptr(ws), ws.numel(), ctypes.c_void_p(s.cuda_stream)),
           "ls_workspace_init")


def ls_workspace_check(ws: torch.Tensor, stream=None) -> int:
    """The workspace's error bits (0: no call on it gave up a wait since it was last
    initialised).  Waits for `stream` (default: the current stream)."""
    _require_gpu(ws)
    s = stream if stream is not None else torch.cuda.current_stream(ws.device)
    flags = ctypes.c_uint32(0)
    st = load_library().ls_workspace_check(_ptr(ws), ctypes.byref(flags), ctypes.c_void_p(s.cuda_stream))
    if st not in (LS_OK, LS_ERR_INCOMPLETE):
        _check(st, "ls_workspace_check")
    return flags.value


_capture_status, _capture_number = ctypes.c_int(0), ctypes.c_ulonglong(0)
_capture_refs = ctypes.byref(_capture_status), ctypes.byref(_capture_number)


def _capture_of(handle: int) -> int | None:
    """The number of the capture that a stream is in; None while it is in none.  Under _ws_lock."""
    if handle == 0:  # the null stream cannot be captured
        return None
    if (_lib or load_library()).hipStreamGetCaptureInfo(handle, *_capture_refs) != 0:
        raise LibscanError(LS_ERR_HIP, "hipStreamGetCaptureInfo")
    return _capture_number.value if _capture_status.value else None


def _new_workspace(device: torch.device, stream: torch.cuda.Stream, nbytes: int,
                   fill: int | None = None) -> torch.Tensor:
    """A workspace whose first `fill` bytes (None: all) are zero."""
    with torch.cuda.stream(stream):  # while it is being captured: from the graph's pool
        new = torch.empty((max(nbytes, 1 << 16) + 255) & ~255, dtype=torch.uint8, device=device)
    ls_workspace_init(new[:fill], stream)
    return new


def _graph_workspace(device: torch.device, stream: torch.cuda.Stream, nbytes: int, kind: str,
                     key: tuple, capture: int) -> torch.Tensor:
    """The workspace of the graph that is being captured on `stream`, for no other graph
    and no eager call: these could run between or beside its replays."""
    last, buf = _ws_graph.get(key, (None, None))
    if last != capture or buf.numel() < nbytes:
        buf = _ws_cache.get(key)
        if buf is not None and buf.numel() >= nbytes and \
                buf.numel() + sum(ws.numel() for _, ws in _ws_retired) <= WORKSPACES_TAKEN_BYTES:
            # filled by an eager call, and not used by one again
            _ws_retired.append((key, _ws_cache.pop(key)))
            _ws_uses.pop(key, None)
        else:
            # the fill is a node of this graph, so only this graph may count on it; plain scratch needs
            # none but its header's error word
            buf = _new_workspace(device, stream, nbytes, None if kind in ("status", "sample") else 256)
        _ws_graph[key] = (capture, buf)
    return buf


def workspace_for(device: torch.device, stream: torch.cuda.Stream, nbytes: int,
                  kind: str = "status") -> torch.Tensor:
    """The cached, initialised uint8 workspace of (device, stream, kind), of at least
    nbytes.  Kinds keep apart what the C ABI requires to be apart: "status" for the
    single-pass scans, segmented scans and compactions (tile status words that must
    never be overwritten with other data), "sort" for the radix sort, "phases"
    for the three-phase scan_ex schemes (plain scratch) and "sample" for
    sample_tokens.  While the stream is being captured, the workspace is that graph's own."""
    with _ws_lock:
        handle = stream.cuda_stream
        key = (device.index, handle, kind)
        if handle != 0:
            capture = _capture_of(handle)
            if capture is not None:
                return _graph_workspace(device, stream, nbytes, kind, key, capture)
        buf = _ws_cache.get(key)
        if buf is None or buf.numel() < nbytes:
            if buf is not None:
                # at least twice the old one while small, so that needs that grow call by call (a row more
                # each time) make few of them.  The old one has no graph to serve (_graph_workspace) and goes
                # back to the stream's memory
                nbytes = max(nbytes, min(2 * buf.numel(), WORKSPACE_DOUBLING_BYTES))
            buf = _ws_cache[key] = _new_workspace(device, stream, nbytes)
            _ws_uses[key] = 0
        elif kind == "status":
            # status words compare epochs modulo 2^26: zero the workspace again well
            # before that many calls (one fill kernel per 2^25 calls)
            _ws_uses[key] = _ws_uses.get(key, 0) + 1
            if _ws_uses[key] >= STATUS_REINIT_CALLS:
                ls_workspace_init(buf, stream)
                _ws_uses[key] = 0
        return buf


def workspace_error_flags(device=None, stream=None) -> int:
    """Error bits of the cached workspace of (device, stream) (defaults: cuda:0's
    current stream) and of those that graphs captured there have taken, the last such
    graph's in any case (once it has been replayed); 0 when there is none yet.  Waits for
    the stream; wait for the graphs' replays before."""
    device = torch.device(device if device is not None else "cuda:0")
    s = stream if stream is not None else torch.cuda.current_stream(device)
    key = (device.index, s.cuda_stream, "status")
    with _ws_lock:
        held = [_ws_cache.get(key), _ws_graph.get(key, (None, None))[1]]
        held += [ws for taken, ws in _ws_retired if taken == key and ws is not held[1]]
        flags = 0
        for ws in held:
            flags |= 0 if ws is None else ls_workspace_check(ws, s)
    return flags


def release_workspaces() -> None:
    """Drop every cached workspace and those given to graphs (no graph that used one may be
    replayed afterwards)."""
    _ws_cache.clear()
    _ws_graph.clear()
    _ws_retired.clear()
    _ws_uses.clear()


def _after_call(ws: torch.Tensor, stream, where: str) -> None:
    """Checked mode: report a call whose bounded wait gave up."""
    if not _checked:
        return
    flags = ls_workspace_check(ws, stream)
    if flags:
        ls_workspace_init(ws, stream)
        raise LibscanError(LS_ERR_INCOMPLETE, f"{where} (workspace error bits {flags:#x})")


def _dtype_of(x: torch.Tensor) -> str:
    try:
        return _TORCH_DTYPES[x.dtype]
    except KeyError:
        raise TypeError(f"libscan: unsupported dtype {x.dtype} (int32, uint32, float32)") from None


def _require_gpu(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libscan: tensors must be on a GPU device")


def _stream_handle(device) -> tuple:
    s = torch.cuda.current_stream(device)
    return s, ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# ------------------------------------------------------------ entry points

def _scan(name: str, x: torch.Tensor, op: str, out, total):
    lib = load_library()
    _require_gpu(x, out, total)
    if not x.is_contiguous():
        raise ValueError("libscan: input must be contiguous")
    dt = _dtype_of(x)
    if out is None:
        out = torch.empty_like(x)
    if out.dtype != x.dtype or out.numel() != x.numel() or not out.is_contiguous():
        raise ValueError("libscan: out must be a contiguous tensor like the input")
    if total is not None and (total.dtype != x.dtype or total.numel() < 1):
        raise ValueError("libscan: total must hold one element of the input dtype")
    n = x.numel()
    stream, sh = _stream_handle(x.device)
    need = ls_scan_workspace_bytes(n, dt, op)
    with _ws_lock:
        ws = workspace_for(x.device, stream, need)
        st = getattr(lib, name)(_ptr(x), _ptr(out), n, DTYPE_CODES[dt], OP_CODES[op], _ptr(total),
                                _ptr(ws), ws.numel(), sh)
        _check(st, name)
        _after_call(ws, stream, name)
    return out


def ls_segmented_workspace_bytes(n: int, dtype: str = "int32", op: str = "sum") -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().ls_segmented_workspace_bytes(n, DTYPE_CODES[dtype], OP_CODES[op],
                                                       ctypes.byref(out)), "ls_segmented_workspace_bytes")
    return out.value


def segmented_scan(x: torch.Tensor, op: str = "sum", exclusive: bool = False,
                   heads: torch.Tensor | None = None, offsets: torch.Tensor | None = None,
                   out: torch.Tensor | None = None, total: torch.Tensor | None = None) -> torch.Tensor:
    """Scan each segment of the flattened x on its own.  Segments by `heads` (n bytes,
    nonzero = first element of a segment; element 0 always starts one) or by
    `offsets` (int64 CSR offsets, nseg + 1 entries from 0 to n); exactly one of the
    two.  total (optional, one element): the inclusive value of the last element."""
    lib = load_library()
    _require_gpu(x, heads, offsets, out, total)
    if (heads is None) == (offsets is None):
        raise ValueError("libscan: give exactly one of heads and offsets")
    if not x.is_contiguous():
        raise ValueError("libscan: input must be contiguous")
    dt = _dtype_of(x)
    n = x.numel()
    if out is None:
        out = torch.empty_like(x)
    if out.dtype != x.dtype or out.numel() != n or not out.is_contiguous():
        raise ValueError("libscan: out must be a contiguous tensor like the input")
    if total is not None and (total.dtype != x.dtype or total.numel() < 1):
        raise ValueError("libscan: total must hold one element of the input dtype")
    stream, sh = _stream_handle(x.device)
    with _ws_lock:
        ws = workspace_for(x.device, stream, ls_segmented_workspace_bytes(n, dt, op))
        excl = 1 if exclusive else 0
        if heads is not None:
            heads = _flags_tensor(heads, n)
            st = lib.segmented_scan(_ptr(x), _ptr(out), n, DTYPE_CODES[dt], OP_CODES[op], excl, _ptr(heads),
                                    _ptr(total), _ptr(ws), ws.numel(), sh)
            _check(st, "segmented_scan")
            _after_call(ws, stream, "segmented_scan")
        else:
            if offsets.dtype != torch.int64 or not offsets.is_contiguous() or offsets.numel() < 1:
                raise ValueError("libscan: offsets must be a contiguous int64 tensor of nseg + 1 entries")
            st = lib.segmented_scan_offsets(_ptr(x), _ptr(out), n, DTYPE_CODES[dt], OP_CODES[op], excl,
                                            _ptr(offsets), offsets.numel() - 1, _ptr(total), _ptr(ws),
                                            ws.numel(), sh)
            _check(st, "segmented_scan_offsets")
            _after_call(ws, stream, "segmented_scan_offsets")
    return out


def scan_inclusive(x: torch.Tensor, op: str = "sum", out: torch.Tensor | None = None,
                   total: torch.Tensor | None = None) -> torch.Tensor:
    """out[i] = x[0] (+) ... (+) x[i] over the flattened tensor; total (optional,
    one element) receives the reduction of all of x.  out may be x (in place)."""
    return _scan("scan_inclusive", x, op, out, total)


def scan_exclusive(x: torch.Tensor, op: str = "sum", out: torch.Tensor | None = None,
                   total: torch.Tensor | None = None) -> torch.Tensor:
    """out[0] = identity, out[i] = x[0] (+) ... (+) x[i-1]."""
    return _scan("scan_exclusive", x, op, out, total)


def scan_noalloc(x: torch.Tensor, op: str = "sum", exclusive: bool = False,
                 out: torch.Tensor | None = None, total: torch.Tensor | None = None) -> torch.Tensor:
    """The scan on the library's fixed per-GPU workspace (no workspace argument, no
    allocation inside the call; n <= LS_SCAN_NOALLOC_MAX_N).  Calls that may overlap
    on one GPU race: keep them on one stream.  With out and total given, this
    function allocates nothing either."""
    lib = load_library()
    _require_gpu(x, out, total)
    if not x.is_contiguous():
        raise ValueError("libscan: input must be contiguous")
    dt = _dtype_of(x)
    if out is None:
        out = torch.empty_like(x)
    if out.dtype != x.dtype or out.numel() != x.numel() or not out.is_contiguous():
        raise ValueError("libscan: out must be a contiguous tensor like the input")
    if total is not None and (total.dtype != x.dtype or total.numel() < 1):
        raise ValueError("libscan: total must hold one element of the input dtype")
    _, sh = _stream_handle(x.device)
    st = lib.scan_noalloc(_ptr(x), _ptr(out), x.numel(), DTYPE_CODES[dt], OP_CODES[op],
                          1 if exclusive else 0, _ptr(total), sh)
    _check(st, "scan_noalloc")
    return out


def scan_ex(x: torch.Tensor, op: str = "sum", inclusive: bool = True,
            scheme: str = "single_pass", out: torch.Tensor | None = None,
            total: torch.Tensor | None = None) -> torch.Tensor:
    """A scan with an explicit device-wide scheme: "single_pass",
    "reduce_then_scan" or "scan_then_propagate" (see ls_scheme in libscan.h)."""
    lib = load_library()
    _require_gpu(x, out, total)
    if not x.is_contiguous():
        raise ValueError("libscan: input must be contiguous")
    dt = _dtype_of(x)
    if out is None:
        out = torch.empty_like(x)
    if out.dtype != x.dtype or out.numel() != x.numel() or not out.is_contiguous():
        raise ValueError("libscan: out must be a contiguous tensor like the input")
    if total is not None and (total.dtype != x.dtype or total.numel() < 1):
        raise ValueError("libscan: total must hold one element of the input dtype")
    n = x.numel()
    stream, sh = _stream_handle(x.device)
    need = ls_scan_ex_workspace_bytes(n, dt, op, scheme)
    phases = scheme in ("reduce_then_scan", "scan_then_propagate")
    with _ws_lock:
        ws = workspace_for(x.device, stream, need, "phases" if phases else "status")
        st = lib.scan_ex(_ptr(x), _ptr(out), n, DTYPE_CODES[dt], OP_CODES[op], 0 if inclusive else 1,
                         SCHEME_CODES[scheme], _ptr(total), _ptr(ws), ws.numel(), sh)
        _check(st, "scan_ex")
        if not phases:  # the three-phase schemes never wait, and keep no error word
            _after_call(ws, stream, "scan_ex")
    return out


def compact_if(x: torch.Tensor, cmp: str, threshold, out: torch.Tensor | None = None,
               count: torch.Tensor | None = None):
    """Stable compaction of the flattened x under (x CMP threshold).

    Returns (out, count): out has x's size, its first `count` cells hold the kept
    elements in input order; count is a one-element int64 device tensor."""
    lib = load_library()
    _require_gpu(x, out, count)
    if not x.is_contiguous():
        raise ValueError("libscan: input must be contiguous")
    dt = _dtype_of(x)
    if out is None:
        out = torch.empty_like(x)
    if count is None:
        count = torch.empty(1, dtype=torch.int64, device=x.device)
    if count.dtype != torch.int64:
        raise ValueError("libscan: count must be int64")
    thr_bits = _threshold_bits(dt, threshold)
    n = x.numel()
    stream, sh = _stream_handle(x.device)
    need = ls_compact_workspace_bytes(n, dt)
    with _ws_lock:
        ws = workspace_for(x.device, stream, need)
        st = lib.compact_if(_ptr(x), _ptr(out), _ptr(count), n, DTYPE_CODES[dt], CMP_CODES[cmp],
                            thr_bits, _ptr(ws), ws.numel(), sh)
        _check(st, "compact_if")
        _after_call(ws, stream, "compact_if")
    return out, count


def _threshold_bits(dt: str, threshold) -> int:
    np_dt = {"int32": "i4", "uint32": "u4", "float32": "f4"}[dt]
    return int(np.array([threshold], dtype=np_dt).view(np.uint32)[0])


def _count_tensor(count, device):
    if count is None:
        count = torch.empty(1, dtype=torch.int64, device=device)
    if count.dtype != torch.int64:
        raise ValueError("libscan: count must be int64")
    return count


def _flags_tensor(flags: torch.Tensor, n: int) -> torch.Tensor:
    if flags.dtype not in (torch.uint8, torch.bool, torch.int8) or flags.numel() != n:
        raise ValueError("libscan: flags must be n bytes (uint8 / bool)")
    if not flags.is_contiguous():
        raise ValueError("libscan: flags must be contiguous")
    return flags


def compact_flags(x: torch.Tensor, flags: torch.Tensor, out: torch.Tensor | None = None,
                  count: torch.Tensor | None = None):
    """Stable compaction of the 32-bit elements of x whose byte flag is nonzero.
    Returns (out, count) like compact_if."""
    lib = load_library()
    _require_gpu(x, flags, out, count)
    if not x.is_contiguous() or x.element_size() != 4:
        raise ValueError("libscan: x must be a contiguous tensor of 32-bit elements")
    n = x.numel()
    flags = _flags_tensor(flags, n)
    if out is None:
        out = torch.empty_like(x)
    count = _count_tensor(count, x.device)
    stream, sh = _stream_handle(x.device)
    with _ws_lock:
        ws = workspace_for(x.device, stream, ls_compact_workspace_bytes(n, "uint32"))
        st = lib.compact_flags(_ptr(x), _ptr(flags), _ptr(out), _ptr(count), n, _ptr(ws), ws.numel(), sh)
        _check(st, "compact_flags")
        _after_call(ws, stream, "compact_flags")
    return out, count


def select_indices_if(x: torch.Tensor, cmp: str, threshold, out: torch.Tensor | None = None,
                      count: torch.Tensor | None = None):
    """Positions (int32 tensor holding uint32 values) of the elements with
    (x CMP threshold), ascending; returns (indices, count)."""
    lib = load_library()
    _require_gpu(x, out, count)
    if not x.is_contiguous():
        raise ValueError("libscan: input must be contiguous")
    dt = _dtype_of(x)
    n = x.numel()
    if out is None:
        out = torch.empty(n, dtype=torch.int32, device=x.device)
    count = _count_tensor(count, x.device)
    stream, sh = _stream_handle(x.device)
    with _ws_lock:
        ws = workspace_for(x.device, stream, ls_compact_workspace_bytes(n, dt))
        st = lib.select_indices_if(_ptr(x), _ptr(out), _ptr(count), n, DTYPE_CODES[dt], CMP_CODES[cmp],
                                   _threshold_bits(dt, threshold), _ptr(ws), ws.numel(), sh)
        _check(st, "select_indices_if")
        _after_call(ws, stream, "select_indices_if")
    return out, count


def select_indices_flags(flags: torch.Tensor, out: torch.Tensor | None = None,
                         count: torch.Tensor | None = None):
    """Positions (int32 tensor holding uint32 values) of the nonzero flag bytes."""
    lib = load_library()
    _require_gpu(flags, out, count)
    n = flags.numel()
    flags = _flags_tensor(flags, n)
    if out is None:
        out = torch.empty(n, dtype=torch.int32, device=flags.device)
    count = _count_tensor(count, flags.device)
    stream, sh = _stream_handle(flags.device)
    with _ws_lock:
        ws = workspace_for(flags.device, stream, ls_compact_workspace_bytes(n, "uint32"))
        st = lib.select_indices_flags(_ptr(flags), _ptr(out), _ptr(count), n, _ptr(ws), ws.numel(), sh)
        _check(st, "select_indices_flags")
        _after_call(ws, stream, "select_indices_flags")
    return out, count


def batched_row_scan(x: torch.Tensor, op: str = "sum", exclusive: bool = True,
                     out: torch.Tensor | None = None) -> torch.Tensor:
    """Scan each row of a contiguous 2-D tensor independently (no carry between rows)."""
    lib = load_library()
    _require_gpu(x, out)
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("libscan: batched_row_scan wants a contiguous 2-D tensor")
    dt = _dtype_of(x)
    if out is None:
        out = torch.empty_like(x)
    rows, cols = x.shape
    _, sh = _stream_handle(x.device)
    st = lib.batched_row_scan(_ptr(x), _ptr(out), rows, cols, DTYPE_CODES[dt], OP_CODES[op],
                              1 if exclusive else 0, sh)
    _check(st, "batched_row_scan")
    return out


def batched_row_scan_ex(x: torch.Tensor, op: str = "sum", exclusive: bool = True,
                        block_scan: str = "wave_dpp", out: torch.Tensor | None = None) -> torch.Tensor:
    """batched_row_scan with an explicit block-level scan: "wave_dpp",
    "hillis_steele", "hillis_steele_double" or "blelloch" (see ls_block_scan)."""
    lib = load_library()
    _require_gpu(x, out)
    if x.dim() != 2 or not x.is_contiguous():
        raise ValueError("libscan: batched_row_scan wants a contiguous 2-D tensor")
    dt = _dtype_of(x)
    if out is None:
        out = torch.empty_like(x)
    rows, cols = x.shape
    _, sh = _stream_handle(x.device)
    st = lib.batched_row_scan_ex(_ptr(x), _ptr(out), rows, cols, DTYPE_CODES[dt], OP_CODES[op],
                                 1 if exclusive else 0, BLOCK_SCAN_CODES[block_scan], sh)
    _check(st, "batched_row_scan_ex")
    return out


def ls_radix_sort_workspace_bytes(n: int, dtype: str, with_values: bool) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().ls_radix_sort_workspace_bytes(n, DTYPE_CODES[dtype], 1 if with_values else 0,
                                                        ctypes.byref(out)),
           "ls_radix_sort_workspace_bytes")
    return out.value


def radix_sort(keys: torch.Tensor, values: torch.Tensor | None = None,
               out_keys: torch.Tensor | None = None, out_values: torch.Tensor | None = None):
    """Stable ascending sort of a flat 32-bit key tensor (int32 / uint32 / float32 in
    IEEE total order), with optional 32-bit values.  Returns (keys, values or None)."""
    lib = load_library()
    _require_gpu(keys, values, out_keys, out_values)
    if not keys.is_contiguous() or (values is not None and not values.is_contiguous()):
        raise ValueError("libscan: keys and values must be contiguous")
    dt = _dtype_of(keys)
    n = keys.numel()
    if values is not None and (values.numel() != n or values.element_size() != 4):
        raise ValueError("libscan: values must hold n 32-bit elements")
    if out_keys is None:
        out_keys = torch.empty_like(keys)
    if values is not None and out_values is None:
        out_values = torch.empty_like(values)
    stream, sh = _stream_handle(keys.device)
    need = ls_radix_sort_workspace_bytes(n, dt, values is not None)
    with _ws_lock:
        ws = workspace_for(keys.device, stream, need, "sort")
        st = lib.radix_sort(_ptr(keys), _ptr(out_keys), _ptr(values), _ptr(out_values), n, DTYPE_CODES[dt],
                            _ptr(ws), ws.numel(), sh)
        _check(st, "radix_sort")
        _after_call(ws, stream, "radix_sort")
    return out_keys, (out_values if values is not None else None)


# ------------------------------------------------------------ a decoding step

# A step makes these calls many times a second, each for a few microseconds of GPU work, so
# an entry point asks all it wants of its tensors in one expression, and goes through them
# one by one (_vector) only to name what is wrong: 10 us a call with
# torch.cuda.current_stream and a helper per tensor, 6 us so, of which 4 are the launch.

def _vector(t, name: str, dtype, n: int, index: int) -> None:
    """Raises unless t is a contiguous vector of n elements of `dtype` on GPU `index`."""
    _require_gpu(t)
    if t.get_device() != index:
        raise ValueError(f"libscan: {name} is on {t.device}, not on cuda:{index}")
    if t.dtype is not dtype:
        raise TypeError(f"libscan: {name} must be {dtype}, not {t.dtype}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"libscan: {name} must be a contiguous vector of {n} elements")


def _matrix(t, name: str, overlapping: bool) -> tuple:
    """(rows, columns, row stride) of a matrix whose rows are contiguous.  Rows may be
    one and the same (stride 0) only where `overlapping`."""
    if not t.is_cuda:
        _require_gpu(t)
    if t.dim() != 2:
        raise ValueError(f"libscan: {name} must be a matrix")
    rows, columns = t.shape
    if t.is_contiguous():
        return rows, columns, columns
    stride, step = t.stride()
    if columns > 1 and step != 1:
        raise ValueError(f"libscan: the rows of {name} must be contiguous")
    if rows > 1 and stride < columns and not (overlapping and stride == 0):
        raise ValueError(f"libscan: the rows of {name} overlap")
    return rows, columns, stride if rows > 1 else columns


def _table(tables, overlapping: bool) -> tuple:
    """(requests, columns, row stride) of a block table."""
    if tables.dtype is not torch.int32:
        raise TypeError(f"libscan: tables must be torch.int32, not {tables.dtype}")
    if tables.is_cuda and tables.dim() == 2 and tables.is_contiguous():
        requests, columns = tables.shape
        return requests, columns, columns
    return _matrix(tables, "tables", overlapping)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:  # pragma: no cover - a torch build without it
    def _raw_stream(index: int) -> int:
        return torch.cuda.current_stream(index).cuda_stream
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


_I32, _I64, _F32, _BOOL = torch.int32, torch.int64, torch.float32, torch.bool


def ls_sample_workspace_bytes(rows: int, vocab: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load_library().ls_sample_workspace_bytes(rows, vocab, ctypes.byref(out)), "ls_sample_workspace_bytes")
    return out.value


def sample_tokens(logits: torch.Tensor, uniforms: torch.Tensor, temperature: torch.Tensor,
                  top_k: torch.Tensor | None = None, top_p: torch.Tensor | None = None,
                  min_p: torch.Tensor | None = None, out: torch.Tensor | None = None,
                  logprobs: torch.Tensor | None = None):
    """One token from each row of logits (rows x vocab; float32, float16 or bfloat16;
    rows contiguous, at any stride), by the row's random number in [0, 1).

    A token's weight is exp((x - max) / temperature).  top_k keeps the k largest logits
    (equal ones: the lower index first; k <= 0 keeps all), top_p of those the smallest
    number whose weights reach top_p of their sum, min_p of those the ones that have at
    least min_p of the largest weight.  The token is the first index at which the running
    sum of the kept weights exceeds uniform * their sum; sums are in 64 bits.
    temperature <= 0 takes the first largest logit.  -inf and NaN are masked; a row with
    nothing left gives token -1 and log-probability -inf.

    uniforms, temperature, top_p, min_p are float32 and top_k int32 vectors of one entry
    a row; a cut that is None is not made.  Returns (tokens int64, logprobs float32),
    written into `out` and `logprobs` where given."""
    lib = _lib or load_library()
    rows, vocab, stride = _matrix(logits, "logits", True)
    code = LOGITS_CODES.get(logits.dtype)
    if code is None:
        raise TypeError(f"libscan: unsupported dtype {logits.dtype} (float32, float16, bfloat16)")
    index = logits.get_device()
    if _current_device() != index:
        with torch.cuda.device(index):
            return sample_tokens(logits, uniforms, temperature, top_k, top_p, min_p, out, logprobs)
    if out is None:
        out = torch.empty(rows, dtype=torch.int64, device=logits.device)
    if logprobs is None:
        logprobs = torch.empty(rows, dtype=torch.float32, device=logits.device)
    one = (rows,)
    if not (uniforms.dtype is _F32 and temperature.dtype is _F32 and out.dtype is _I64 and logprobs.dtype is _F32
            and index == uniforms.get_device() == temperature.get_device() == out.get_device() == logprobs.get_device()
            and one == uniforms.shape == temperature.shape == out.shape == logprobs.shape
            and uniforms.is_contiguous() and temperature.is_contiguous() and out.is_contiguous()
            and logprobs.is_contiguous()):
        for t, name, dtype in ((uniforms, "uniforms", _F32), (temperature, "temperature", _F32), (out, "out", _I64),
                               (logprobs, "logprobs", _F32)):
            _vector(t, name, dtype, rows, index)
    for t, name, dtype in ((top_k, "top_k", _I32), (top_p, "top_p", _F32), (min_p, "min_p", _F32)):
        if t is not None and not (t.dtype is dtype and t.get_device() == index and t.shape == one and t.is_contiguous()):
            _vector(t, name, dtype, rows, index)
    with _ws_lock:
        ws = _sample_workspace(index, rows, vocab)
        st = lib.sample_tokens(
            logits.data_ptr(), rows, vocab, stride, code, uniforms.data_ptr(), temperature.data_ptr(),
            None if top_k is None else top_k.data_ptr(), None if top_p is None else top_p.data_ptr(),
            None if min_p is None else min_p.data_ptr(), out.data_ptr(), logprobs.data_ptr(), ws.data_ptr(), ws.numel(),
            _raw_stream(index))
    if st != LS_OK:
        raise LibscanError(st, "sample_tokens")
    return out, logprobs


def _sample_workspace(index: int, rows: int, vocab: int) -> torch.Tensor:
    """The current stream's workspace for sample_tokens (workspace_for's, found sooner)."""
    need, handle = ls_sample_workspace_bytes(rows, vocab), _raw_stream(index)
    buf = _ws_cache.get((index, handle, "sample"))
    if buf is None or buf.numel() < need or (handle != 0 and _capture_of(handle) is not None):
        device = torch.device("cuda", index)
        buf = workspace_for(device, torch.cuda.current_stream(device), need, "sample")
    return buf


def pages_append(lens: torch.Tensor, new_lens: torch.Tensor, tables: torch.Tensor, free_pages: torch.Tensor,
                 free_count: torch.Tensor, page_size: int, count_out: torch.Tensor | None = None,
                 granted: torch.Tensor | None = None):
    """Gives each request the pages that new_lens more tokens need, into its row of
    `tables` (int32, requests x columns), from the end of the free list (the first
    free_count entries of free_pages).  Requests are served in order; from the first one
    that the free list cannot serve, only requests that need no page are granted, and a
    request that needs more columns than the table has is passed over.

    Returns (count_out, granted): free pages left (one int64) and a bool for each
    request.  count_out may not be free_count itself."""
    lib = _lib or load_library()
    requests, columns, stride = _table(tables, False)
    index = tables.get_device()
    if _current_device() != index:
        with torch.cuda.device(index):
            return pages_append(lens, new_lens, tables, free_pages, free_count, page_size, count_out, granted)
    if count_out is None:
        count_out = torch.empty(1, dtype=torch.int64, device=tables.device)
    if granted is None:
        granted = torch.empty(requests, dtype=torch.bool, device=tables.device)
    capacity = free_pages.numel()
    if not 1 <= page_size < 1 << 31:
        raise ValueError("libscan: page_size must be in [1, 2^31)")
    one = (requests,)
    if not (lens.dtype is _I32 and new_lens.dtype is _I32 and free_pages.dtype is _I32 and free_count.dtype is _I64
            and count_out.dtype is _I64 and granted.dtype is _BOOL
            and index == lens.get_device() == new_lens.get_device() == free_pages.get_device()
            == free_count.get_device() == count_out.get_device() == granted.get_device()
            and one == lens.shape == new_lens.shape == granted.shape and free_pages.shape == (capacity,)
            and (1,) == free_count.shape == count_out.shape and lens.is_contiguous() and new_lens.is_contiguous()
            and free_pages.is_contiguous() and granted.is_contiguous()):
        for t, name, dtype, n in ((lens, "lens", _I32, requests), (new_lens, "new_lens", _I32, requests),
                                  (free_pages, "free_pages", _I32, capacity), (free_count, "free_count", _I64, 1),
                                  (count_out, "count_out", _I64, 1), (granted, "granted", _BOOL, requests)):
            _vector(t, name, dtype, n, index)
    st = lib.pages_append(lens.data_ptr(), new_lens.data_ptr(), requests, tables.data_ptr(), columns, stride,
                          free_pages.data_ptr(), capacity, free_count.data_ptr(), page_size, count_out.data_ptr(),
                          granted.data_ptr(), _raw_stream(index))
    if st != LS_OK:
        raise LibscanError(st, "pages_append")
    return count_out, granted


def slot_map(lens: torch.Tensor, new_lens: torch.Tensor, tables: torch.Tensor, page_size: int, capacity: int,
             out: tuple | None = None):
    """Where this step's new tokens go in a paged cache: for each of `capacity` entries
    (tokens in order of request and position) its slot page * page_size + offset (int64;
    -1 where the table holds no page), its position and its request (int32), and the
    requests' offsets (int64, one more than requests).  Entries past the last token get
    slot -1, position 0, request -1.

    Returns (slots, positions, requests, offsets), written into the tensors of `out`
    where given."""
    lib = _lib or load_library()
    requests, columns, stride = _table(tables, True)
    index = tables.get_device()
    if _current_device() != index:
        with torch.cuda.device(index):
            return slot_map(lens, new_lens, tables, page_size, capacity, out)
    if out is None:
        n, device = max(0, capacity), tables.device
        out = (torch.empty(n, dtype=torch.int64, device=device), torch.empty(n, dtype=torch.int32, device=device),
               torch.empty(n, dtype=torch.int32, device=device),
               torch.empty(requests + 1, dtype=torch.int64, device=device))
    slots, positions, ids, offsets = out
    if capacity < 0:
        raise ValueError("libscan: capacity must not be negative")
    if not 1 <= page_size < 1 << 31:
        raise ValueError("libscan: page_size must be in [1, 2^31)")
    one, room = (requests,), (capacity,)
    if not (lens.dtype is _I32 and new_lens.dtype is _I32 and slots.dtype is _I64 and positions.dtype is _I32
            and ids.dtype is _I32 and offsets.dtype is _I64
            and index == lens.get_device() == new_lens.get_device() == slots.get_device()
            == positions.get_device() == ids.get_device() == offsets.get_device()
            and one == lens.shape == new_lens.shape and room == slots.shape == positions.shape == ids.shape
            and offsets.shape == (requests + 1,) and lens.is_contiguous() and new_lens.is_contiguous()
            and slots.is_contiguous() and positions.is_contiguous() and ids.is_contiguous()
            and offsets.is_contiguous()):
        for t, name, dtype, n in ((lens, "lens", _I32, requests), (new_lens, "new_lens", _I32, requests),
                                  (slots, "slots", _I64, capacity), (positions, "positions", _I32, capacity),
                                  (ids, "requests", _I32, capacity), (offsets, "offsets", _I64, requests + 1)):
            _vector(t, name, dtype, n, index)
    st = lib.slot_map(lens.data_ptr(), new_lens.data_ptr(), requests, tables.data_ptr(), columns, stride, page_size,
                      capacity, slots.data_ptr(), positions.data_ptr(), ids.data_ptr(), offsets.data_ptr(),
                      _raw_stream(index))
    if st != LS_OK:
        raise LibscanError(st, "slot_map")
    return slots, positions, ids, offsets


def pages_release(lens: torch.Tensor, finished: torch.Tensor, tables: torch.Tensor, free_pages: torch.Tensor,
                  free_count: torch.Tensor, page_size: int, count_out: torch.Tensor | None = None) -> torch.Tensor:
    """Puts the pages of the finished requests (a bool each) back on the free list, behind
    its free_count entries, in order of request and column.  Returns count_out: the new
    number of free pages (one int64; not free_count itself)."""
    lib = _lib or load_library()
    requests, columns, stride = _table(tables, True)
    index = tables.get_device()
    if _current_device() != index:
        with torch.cuda.device(index):
            return pages_release(lens, finished, tables, free_pages, free_count, page_size, count_out)
    if count_out is None:
        count_out = torch.empty(1, dtype=torch.int64, device=tables.device)
    capacity = free_pages.numel()
    if not 1 <= page_size < 1 << 31:
        raise ValueError("libscan: page_size must be in [1, 2^31)")
    one = (requests,)
    if not (lens.dtype is _I32 and finished.dtype is _BOOL and free_pages.dtype is _I32 and free_count.dtype is _I64
            and count_out.dtype is _I64
            and index == lens.get_device() == finished.get_device() == free_pages.get_device()
            == free_count.get_device() == count_out.get_device()
            and one == lens.shape == finished.shape and free_pages.shape == (capacity,)
            and (1,) == free_count.shape == count_out.shape and lens.is_contiguous() and finished.is_contiguous()
            and free_pages.is_contiguous()):
        for t, name, dtype, n in ((lens, "lens", _I32, requests), (finished, "finished", _BOOL, requests),
                                  (free_pages, "free_pages", _I32, capacity), (free_count, "free_count", _I64, 1),
                                  (count_out, "count_out", _I64, 1)):
            _vector(t, name, dtype, n, index)
    st = lib.pages_release(lens.data_ptr(), finished.data_ptr(), requests, tables.data_ptr(), columns, stride,
                           free_pages.data_ptr(), capacity, free_count.data_ptr(), page_size, count_out.data_ptr(),
                           _raw_stream(index))
    if st != LS_OK:
        raise LibscanError(st, "pages_release")
    return count_out
