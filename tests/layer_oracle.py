"""The gated recurrence and the experts' rows, written from their definitions in 64 bits with
numpy, a token after the other.  They share no code with the library.

recurrence() and gradients() also give how far float32 may be off.  Let u = 2^-24, the
rounding of one float32 operation.  A decay carries c u: exp2 and the reciprocal are right to
an ulp (2 u each), the argument g log2(e) is rounded (|g| u of exp2's result), 1 + e and e r
once each: c = 8 + |g| covers them; a decay given directly has none.  b = x or (1 - a) x
carries the same.  A value that a token put in d tokens ago has gone through d products and
d additions, whatever their order, so it is off by at most (c + 2)(d + 1) u, and another few for
the joins of waves and tiles (8 u is taken; each join is a product and an addition, and
their number is part of d).  With S_t the sum of the magnitudes of what is in h_t and W_t the same
weighted by the ages, the bound is u (c + 2) (W_t + 9 S_t): both are recurrences themselves."""
import numpy as np

U = 2.0**-24


def decay(gate, gating):
    g = np.asarray(gate, dtype=np.float64)
    if gating == "decay":
        return g, 2.0
    with np.errstate(over="ignore"):
        a = np.exp(g) if gating == "log" else 1 / (1 + np.exp(-g))
    finite = np.abs(g[np.isfinite(g)])
    return a, 10.0 + float(finite.max(initial=0.0))


def rest_of(gate):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(np.asarray(gate, dtype=np.float64)))


def recurrence(x, gate, state, gating):
    """(h, bound of |float32 h - h|, final state) of sequences x tokens x channels."""
    x = np.asarray(x, dtype=np.float64)
    a, c = decay(gate, gating)
    b = rest_of(gate) * x if gating == "sigmoid" else x
    batch, length, channels = x.shape
    now = np.zeros((batch, channels)) if state is None else np.asarray(state, dtype=np.float64).copy()
    size, aged = np.abs(now), np.zeros_like(now)
    h, bound = np.empty_like(x), np.empty_like(x)
    for t in range(length):
        now = a[:, t] * now + b[:, t]
        m = np.abs(a[:, t])
        aged = m * (aged + size)
        size = m * size + np.abs(b[:, t])
        h[:, t], bound[:, t] = now, U * c * (aged + 9 * size)
    return h, bound, now


def gradients(x, gate, state, dout, dstate_out, gating):
    """(dx, dgate, dstate) and the bounds of what float32 may be off."""
    x, dout = np.asarray(x, dtype=np.float64), np.asarray(dout, dtype=np.float64)
    a, c = decay(gate, gating)
    rest = rest_of(gate)
    h, hbound, _ = recurrence(x, gate, state, gating)
    batch, length, channels = x.shape
    first = np.zeros((batch, channels)) if state is None else np.asarray(state, dtype=np.float64)
    mu = np.zeros((batch, channels)) if dstate_out is None else np.asarray(dstate_out, dtype=np.float64).copy()
    size, aged = np.abs(mu), np.zeros_like(mu)
    dx, dg, ex, eg = (np.empty_like(x) for _ in range(4))
    for t in reversed(range(length)):
        lam = dout[:, t] + mu
        size, aged = size + np.abs(dout[:, t]), aged + size
        elam = U * c * (aged + 9 * size)
        before = h[:, t - 1] if t else first
        ebefore = hbound[:, t - 1] if t else np.zeros_like(first)
        at = a[:, t]
        if gating == "sigmoid":
            r = rest[:, t]
            dx[:, t] = lam * r
            ex[:, t] = (elam + 2 * c * U * np.abs(lam)) * r
            gap = before - x[:, t]
            dg[:, t] = lam * gap * at * r
            eg[:, t] = at * r * (np.abs(gap) * (elam + 4 * c * U * np.abs(lam)) + np.abs(lam) * (ebefore + U * np.abs(gap)))
        else:
            dx[:, t], ex[:, t] = lam, elam
            k = at if gating == "log" else 1.0
            dg[:, t] = lam * before * k
            eg[:, t] = np.abs(k) * (np.abs(before) * (elam + 2 * c * U * np.abs(lam)) + np.abs(lam) * ebefore)
        mu = at * lam
        size, aged = np.abs(at) * size, np.abs(at) * aged
    return (dx, dg, mu), (ex, eg, U * c * (aged + 9 * size))


def packed(fn, offsets, *args):
    """fn of each non-empty sequence alone: a list of (sequence, first row, last row + 1, result)."""
    out = []
    for s in range(len(offsets) - 1):
        lo, hi = int(offsets[s]), int(offsets[s + 1])
        if hi > lo:
            rows = [None if v is None else (v[lo:hi][None] if whole else v[s:s + 1]) for v, whole in args]
            out.append((s, lo, hi, fn(*rows)))
    return out


def sort(experts, num_experts):
    """(offsets, order, places) of flat pairs, one pair after the other."""
    lists = [[] for _ in range(num_experts)]
    for p, e in enumerate(np.asarray(experts).reshape(-1).tolist()):
        if 0 <= e < num_experts:
            lists[e].append(p)
    order = np.full(np.asarray(experts).size, -1, dtype=np.int32)
    places = order.copy()
    flat = [p for l in lists for p in l]
    order[: len(flat)] = flat
    places[flat] = np.arange(len(flat))
    return np.concatenate([[0], np.cumsum([len(l) for l in lists])]), order, places.reshape(np.shape(experts))


def gather(x, places, rows):
    rows = np.array(rows)
    for t, j in np.ndindex(*places.shape):
        if 0 <= places[t, j] < len(rows):
            rows[places[t, j]] = x[t]
    return rows


def combine(rows, places, weights):
    """(sums, sums of magnitudes)"""
    rows = np.asarray(rows, dtype=np.float64)
    out, size = np.zeros((places.shape[0], rows.shape[1])), np.zeros((places.shape[0], rows.shape[1]))
    for t, j in np.ndindex(*places.shape):
        if 0 <= places[t, j] < len(rows):
            part = rows[places[t, j]] * (1.0 if weights is None else float(weights[t, j]))
            out[t] += part
            size[t] += np.abs(part)
    return out, size


def combine_backward(dout, rows, places, weights, drows):
    """(drows, dweights, sums of magnitudes of dweights)"""
    dout, rows = np.asarray(dout, dtype=np.float64), np.asarray(rows, dtype=np.float64)
    drows = np.array(drows, dtype=np.float64)
    dw, size = np.zeros(places.shape), np.zeros(places.shape)
    for t, j in np.ndindex(*places.shape):
        at = places[t, j]
        if 0 <= at < len(rows):
            drows[at] = dout[t] * float(weights[t, j])
            dw[t, j] = np.dot(dout[t], rows[at])
            size[t, j] = np.abs(dout[t] * rows[at]).sum()
    return drows, dw, size
