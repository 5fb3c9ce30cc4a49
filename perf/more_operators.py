"""The operators of a layer with a gated recurrence and experts, as measured cases.

recur        the gated linear recurrence over sequences, packed rows or one token each (ps.gated_recurrence)
train        the recurrence and its gradients (ps.gated_recurrence, ps.gated_recurrence_backward)
dispatch     tokens to the rows of their experts (ps.experts_sort, ps.experts_gather)
combine      the experts' rows back to their tokens, weighted (ps.experts_combine)
back         the gradients of combine and dispatch (ps.experts_combine_backward, ps.experts_combine)

A case is a dict of plain values; listed() and draw() make them, prepare() makes the
tensors a program holds before the call, run() is the call itself: in elementary torch
operations where `own` is false, with the library where it is true.
"""
import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one chat, one token: latency is what counts
        dict(name="recur-step-1", op="recur", batch=1, length=1, channels=2048, dtype="bfloat16", gating="sigmoid",
             packed=False, state=True, fused=True),
        # a decoding step of a full batch
        dict(name="recur-step-256", op="recur", batch=256, length=1, channels=4096, dtype="bfloat16", gating="sigmoid",
             packed=False, state=True, fused=True),
        # prompts in chunks among decoding requests and idle ones, in a buffer of fixed length
        dict(name="recur-packed-96", op="recur", batch=96, length=200, channels=2560, dtype="float16", gating="sigmoid",
             packed=True, state=True, fused=True),
        # one long document
        dict(name="recur-long-65536", op="recur", batch=1, length=65536, channels=2048, dtype="bfloat16", gating="log",
             packed=False, state=False, fused=False),
        # a training step's layer
        dict(name="train-4x4096", op="train", batch=4, length=4096, channels=2048, dtype="bfloat16", gating="sigmoid",
             packed=False, state=False, fused=True),
        # odd sizes in full precision, the state handed from piece to piece of a sequence
        dict(name="train-odd", op="train", batch=3, length=1777, channels=1001, dtype="float32", gating="decay",
             packed=False, state=True, fused=False),
        # a decoding step's tokens to their experts
        dict(name="dispatch-32", op="dispatch", tokens=32, top=8, experts=128, channels=4096, dtype="bfloat16",
             dropped=0.0),
        # a wave of prompts
        dict(name="dispatch-16384", op="dispatch", tokens=16384, top=8, experts=256, channels=2048, dtype="bfloat16",
             dropped=0.0),
        # a small odd batch, some pairs over their expert's capacity
        dict(name="combine-61", op="combine", tokens=61, top=6, experts=160, channels=5120, dtype="float16",
             dropped=0.1),
        # prompts or a training batch
        dict(name="combine-8192", op="combine", tokens=8192, top=8, experts=64, channels=4096, dtype="bfloat16",
             dropped=0.0),
        # odd sizes in full precision
        dict(name="back-odd", op="back", tokens=777, top=3, experts=17, channels=1023, dtype="float32", dropped=0.05),
        # a training batch
        dict(name="back-8192", op="back", tokens=8192, top=4, experts=64, channels=4096, dtype="bfloat16", dropped=0.0),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["recur", "recur", "train", "dispatch", "combine", "back"])
    dtype = rng.choice(["float32", "float16", "bfloat16"])
    channels = _log_int(rng, 64, 8192)
    if rng.random() < 0.6:
        channels = max(64, channels // 64 * 64)
    if op in ("recur", "train"):
        room = ((1 << 26) if op == "recur" else (1 << 24)) // channels
        packed = op == "recur" and rng.random() < 0.4
        length = 1 if op == "recur" and not packed and rng.random() < 0.3 else _log_int(rng, 2, min(room, 65536))
        batch = _log_int(rng, 1, max(1, min(512, room // length)))
        return dict(op=op, batch=batch, length=length, channels=channels, dtype=dtype,
                    gating=rng.choice(["sigmoid", "log", "decay"]), packed=packed, state=rng.random() < 0.6,
                    fused=rng.random() < 0.5)
    top = rng.randint(1, 10)
    tokens = _log_int(rng, 1, max(1, min(32768, (1 << 26) // (channels * top))))
    return dict(op=op, tokens=tokens, top=top, experts=_log_int(rng, max(2, top), 512), channels=channels, dtype=dtype,
                dropped=rng.choice([0.0, 0.0, rng.uniform(0.02, 0.5)]))


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _gates(shape, gating, dtype, g):
    """Gates as trained layers have them: memories of one to some thousand tokens."""
    z = torch.randn(shape, device=DEV, generator=g)
    if gating == "sigmoid":
        return z * 1.5 + 2.0
    rate = torch.exp(z * 1.5 - 3.5)  # of forgetting, a token
    return -rate if gating == "log" else torch.exp(-rate)


def _packed_rows(case):
    """Room for the tokens of a step, some more than come as a rule."""
    return max(1, int(case["batch"] * (0.3 + 0.35 * (case["length"] + 1)) * 1.1) + 8)


def _recur_inputs(case, seed):
    g = _generator(seed)
    dtype, batch, length, d = DTYPES[case["dtype"]], case["batch"], case["length"], case["channels"]
    shape = (_packed_rows(case),) if case["packed"] else (batch, length)
    if case["fused"]:  # x and gate are halves of one projection's output
        both = torch.empty(*shape, 2 * d, device=DEV, dtype=dtype)
        x, gate = both[..., :d], both[..., d:]
    else:
        x, gate = (torch.empty(*shape, d, device=DEV, dtype=dtype) for _ in range(2))
    x.copy_(torch.randn(x.shape, device=DEV, generator=g))
    gate.copy_(_gates(x.shape, case["gating"], dtype, g))
    s = dict(x=x, gate=gate, gating=case["gating"], state=None, offsets=None, out=None)
    if case["state"]:
        s["state"] = torch.randn(batch, d, device=DEV, generator=g)
    if case["packed"]:
        # two in ten requests are idle, three decode one token, the others hold a piece of their prompt
        kind = torch.rand(batch, device=DEV, generator=g)
        new = torch.randint(1, length + 1, (batch,), device=DEV, generator=g)
        new = torch.where(kind < 0.3, torch.ones_like(new), new)
        new = torch.where(kind > 0.8, torch.zeros_like(new), new)
        ends = torch.cumsum(new, 0).clamp_max(x.shape[0])
        s["offsets"] = torch.cat([torch.zeros_like(ends[:1]), ends])
        s["out"] = torch.zeros(x.shape, device=DEV, dtype=dtype)  # rows behind the last token stay
    if case["op"] == "train":
        s["dout"] = torch.randn(x.shape, device=DEV, generator=g).to(dtype)
        s["dstate_out"] = torch.randn(batch, d, device=DEV, generator=g) if case["state"] else None
    return s


def _route(case, g):
    """A router's choice: experts of unequal popularity, no expert twice for a token."""
    favour = torch.randn(case["experts"], device=DEV, generator=g)
    score = favour + torch.randn(case["tokens"], case["experts"], device=DEV, generator=g) * 1.5
    experts = torch.sort(score, dim=1, descending=True).indices[:, : case["top"]].contiguous()
    drop = torch.rand(experts.shape, device=DEV, generator=g) < case["dropped"]
    return torch.where(drop, torch.full_like(experts, -1), experts)


def _experts_inputs(case, seed):
    g = _generator(seed)
    dtype, tokens, top, d = DTYPES[case["dtype"]], case["tokens"], case["top"], case["channels"]
    normal = lambda *shape: torch.randn(*shape, device=DEV, generator=g).to(dtype)
    experts = _route(case, g)
    if case["op"] == "dispatch":
        return dict(experts=experts, num_experts=case["experts"], x=normal(tokens, d),
                    rows=torch.zeros(tokens * top, d, device=DEV, dtype=dtype))
    places = _plain_sort(experts, case["experts"])[2]
    s = dict(places=places, rows=normal(tokens * top, d),
             weights=torch.softmax(torch.randn(tokens, top, device=DEV, generator=g), 1))
    if case["op"] == "back":
        s["dout"] = normal(tokens, d)
        s["dgathered"] = normal(tokens * top, d)
        s["drows"] = torch.zeros(tokens * top, d, device=DEV, dtype=dtype)
    return s


def prepare(case, seed):
    state = _recur_inputs(case, seed) if case["op"] in ("recur", "train") else _experts_inputs(case, seed)
    state["op"] = case["op"]
    return state


# ------------------------------------------------------------------ plain forms

def _maps(s):
    """The maps h -> a h + b of all tokens, and 1 - a."""
    # copies, also of float32: what follows adds to them in place
    x, g = s["x"].to(torch.float32, copy=True), s["gate"].to(torch.float32, copy=True)
    if s["gating"] == "sigmoid":
        a, rest = 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))
        return a, rest * x, rest
    return (torch.exp(g) if s["gating"] == "log" else g), x, None


def _compose(a, b, dim):
    """Running composition of maps along dim: windows of 1, 2, 4, ... tokens."""
    step, n = 1, a.shape[dim]
    while step < n:
        late, early = a.narrow(dim, step, n - step), b.narrow(dim, 0, n - step)
        b = torch.cat([b.narrow(dim, 0, step), b.narrow(dim, step, n - step) + late * early], dim)
        a = torch.cat([a.narrow(dim, 0, step), late * a.narrow(dim, 0, n - step)], dim)
        step *= 2
    return b


def _plain_recur(s):
    a, b, _ = _maps(s)
    if s["offsets"] is None:
        if s["state"] is not None:
            b[:, 0] += a[:, 0] * s["state"]
        h = _compose(a, b, 1)
        return h.to(s["x"].dtype), h[:, -1].clone()
    first, last = s["offsets"][:-1], s["offsets"][1:]
    some = last > first
    state = s["state"] if s["state"] is not None else torch.zeros(first.numel(), a.shape[1], device=a.device)
    heads = first[some]
    b[heads] += a[heads] * state[some]
    a[heads] = 0
    h = _compose(a, b, 0)
    live = torch.arange(a.shape[0], device=a.device) < last[-1]
    out = torch.where(live[:, None], h.to(s["x"].dtype), s["out"])
    return out, torch.where(some[:, None], h[(last - 1).clamp_min(0)], state)


def _plain_train(s):
    a, b, rest = _maps(s)
    first = s["state"] if s["state"] is not None else torch.zeros_like(a[:, 0])
    b[:, 0] += a[:, 0] * first
    h = _compose(a, b, 1)
    before = torch.cat([first[:, None], h[:, :-1]], 1)
    dout = s["dout"].to(torch.float32, copy=True)
    if s["dstate_out"] is not None:
        dout[:, -1] += s["dstate_out"]
    # from the last token to the first, with the decay of the token behind
    behind = torch.cat([torch.zeros_like(a[:, :1]), a.flip(1)[:, :-1]], 1)
    lam = _compose(behind, dout.flip(1), 1).flip(1)
    if s["gating"] == "sigmoid":
        dx, dgate = lam * rest, lam * (before - s["x"].float()) * a * rest
    else:
        dx, dgate = lam, lam * before * (a if s["gating"] == "log" else 1)
    dtype = s["x"].dtype
    return h.to(dtype), h[:, -1].clone(), dx.to(dtype), dgate.to(dtype), lam[:, 0] * a[:, 0]


def _plain_sort(experts, num_experts):
    flat = experts.reshape(-1)
    key = torch.where((flat >= 0) & (flat < num_experts), flat, torch.full_like(flat, num_experts))
    ordered, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(ordered, torch.arange(num_experts + 1, device=flat.device))
    places = torch.empty_like(order)
    places[order] = torch.arange(flat.numel(), device=flat.device)
    places = torch.where(key < num_experts, places, torch.full_like(places, -1))
    order = torch.where(ordered < num_experts, order, torch.full_like(order, -1))
    return offsets, order.to(torch.int32), places.to(torch.int32).reshape(experts.shape)


def _plain_dispatch(s):
    offsets, order, places = _plain_sort(s["experts"], s["num_experts"])
    token = (order.clamp_min(0) // s["experts"].shape[1]).long()
    rows = torch.where((order >= 0)[:, None], s["x"][token], s["rows"])
    return offsets, order, places, rows


def _plain_combine(rows, places, weights):
    held = rows[places.clamp_min(0).long()].float()
    if weights is not None:
        held = held * weights[:, :, None]
    return torch.where((places >= 0)[:, :, None], held, torch.zeros_like(held)).sum(1)


def _plain_back(s):
    rows, places, weights, dtype = s["rows"], s["places"], s["weights"], s["rows"].dtype
    dout, at, routed = s["dout"].float(), places.clamp_min(0).long(), places >= 0
    dheld = (weights[:, :, None] * dout[:, None]).to(dtype)
    drows = s["drows"].clone()
    drows[places[routed].long()] = dheld[routed]
    dweights = (rows[at].float() * dout[:, None]).sum(2)
    dx = _plain_combine(s["dgathered"], places, None)
    return drows, torch.where(routed, dweights, torch.zeros_like(dweights)), dx.to(dtype)


# ------------------------------------------------------------------ one pass

def run(state):
    s, op = state, state["op"]
    if not own:
        if op == "combine":
            return _plain_combine(s["rows"], s["places"], s["weights"]).to(s["rows"].dtype)
        return {"recur": _plain_recur, "train": _plain_train, "dispatch": _plain_dispatch, "back": _plain_back}[op](s)
    import prefix_scan_stream_amd as ps
    if op == "recur":
        return ps.gated_recurrence(s["x"], s["gate"], state=s["state"], gating=s["gating"], offsets=s["offsets"],
                                   out=s["out"])
    if op == "train":
        carries = ps.recurrence_carries(s["x"])
        h, state_out = ps.gated_recurrence(s["x"], s["gate"], state=s["state"], gating=s["gating"], carries=carries)
        dx, dgate, dstate = ps.gated_recurrence_backward(s["dout"], s["x"], s["gate"], carries, state=s["state"],
                                                         dstate_out=s["dstate_out"], gating=s["gating"])
        return h, state_out, dx, dgate, dstate
    if op == "dispatch":
        offsets, order, places = ps.experts_sort(s["experts"], s["num_experts"])
        return offsets, order, places, ps.experts_gather(s["x"], places, out=s["rows"])
    if op == "combine":
        return ps.experts_combine(s["rows"], s["places"], s["weights"])
    drows, dweights = ps.experts_combine_backward(s["dout"], s["rows"], s["places"], s["weights"], drows=s["drows"])
    return drows, dweights, ps.experts_combine(s["dgathered"], s["places"])


def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    d = case["channels"]
    if case["op"] in ("recur", "train"):
        batch, states = case["batch"], 2 if case["state"] else 1
        # of a packed step, what comes on average
        n = batch * (0.3 + 0.25 * (case["length"] + 1)) if case["packed"] else batch * case["length"]
        # the gate's value 4, the map 2 to 4
        forward = 8 if case["gating"] == "sigmoid" else 6 if case["gating"] == "log" else 2
        if case["op"] == "recur":
            return {"bytes": int(n * d * 3 * size + batch * d * 4 * states), "flops": int(n * d * forward)}
        # x, gate and the gradient of h in; h and the gradients of x and gate out
        return {"bytes": int(n * d * 6 * size + batch * d * 4 * 2 * states), "flops": int(n * d * (forward + 8))}
    tokens, top = case["tokens"], case["top"]
    pairs, held = tokens * top, tokens * top * (1 - case["dropped"])
    if case["op"] == "dispatch":
        return {"bytes": int(pairs * (8 + 8) + 8 * case["experts"] + (tokens + held) * d * size), "flops": int(pairs * 8)}
    if case["op"] == "combine":
        return {"bytes": int(pairs * 8 + (held + tokens) * d * size), "flops": int(2 * held * d)}
    # rows, the gradients of the sums and of the gathered rows in; those of the rows and of the tokens out
    return {"bytes": int(pairs * 12 + (3 * held + 2 * tokens) * d * size), "flops": int(4 * held * d)}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_decay(s):
    g = s["gate"].double()
    return torch.sigmoid(g) if s["gating"] == "sigmoid" else torch.exp(g) if s["gating"] == "log" else g


def _exact_walk(s, a, batch):
    """h of every token, one token after the other (rows of all sequences side by side)."""
    x = s["x"].double()
    put = x - a * x if s["gating"] == "sigmoid" else x
    h = torch.empty_like(put)
    now = s["state"].double() if s["state"] is not None else torch.zeros(batch, x.shape[-1], device=DEV, dtype=torch.float64)
    if s["offsets"] is None:
        for t in range(x.shape[1]):
            torch.addcmul(put[:, t], a[:, t], now, out=h[:, t])
            now = h[:, t]
        return h, now.clone()
    ends = s["offsets"].tolist()
    final = now.clone()
    for r in range(batch):
        for t in range(ends[r], ends[r + 1]):
            torch.addcmul(put[t], a[t], final[r], out=h[t])
            final[r] = h[t]
    h[ends[-1]:] = s["out"][ends[-1]:].double()
    return h, final


def _exact_train(s, batch):
    a = _exact_decay(s)
    h, final = _exact_walk(s, a, batch)
    x, dh = s["x"].double(), s["dout"].double()
    start = s["state"].double() if s["state"] is not None else torch.zeros_like(final)
    mu = s["dstate_out"].double() if s["dstate_out"] is not None else torch.zeros_like(final)
    dx, dgate = torch.empty_like(x), torch.empty_like(x)
    for t in reversed(range(x.shape[1])):
        lam = dh[:, t] + mu
        mu = a[:, t] * lam
        before = h[:, t - 1] if t else start
        if s["gating"] == "sigmoid":
            dx[:, t] = lam - mu
            dgate[:, t] = (before - x[:, t]) * (lam - mu) * a[:, t]
        else:
            dx[:, t] = lam
            dgate[:, t] = before * (mu if s["gating"] == "log" else lam)
    return h, final, dx, dgate, mu


def _exact_experts(s):
    op = s["op"]
    if op == "dispatch":
        experts, top = s["experts"].cpu(), s["experts"].shape[1]
        flat = experts.reshape(-1)
        lists = [torch.nonzero(flat == e)[:, 0] for e in range(s["num_experts"])]
        pairs = torch.cat(lists)
        offsets = torch.tensor([0] + [p.numel() for p in lists]).cumsum(0)
        order = torch.full((flat.numel(),), -1, dtype=torch.int32)
        order[: pairs.numel()] = pairs.int()
        places = torch.full((flat.numel(),), -1, dtype=torch.int32)
        places[pairs] = torch.arange(pairs.numel(), dtype=torch.int32)
        rows = s["rows"].double()
        rows[: pairs.numel()] = s["x"].double()[(pairs // top).to(DEV)]
        return offsets.to(DEV), order.to(DEV), places.reshape(experts.shape).to(DEV), rows
    places, rows, weights = s["places"], s["rows"].double(), s["weights"].double()
    tokens, top = places.shape
    token, choice = torch.nonzero(places >= 0, as_tuple=True)
    row = places[token, choice].long()
    if op == "combine":
        out = torch.zeros(tokens, rows.shape[1], device=DEV, dtype=torch.float64)
        return out.index_add_(0, token, rows[row] * weights[token, choice][:, None])
    drows, dout = s["drows"].double(), s["dout"].double()
    drows[row] = dout[token] * weights[token, choice][:, None]
    dweights = torch.zeros_like(weights)
    dweights[token, choice] = (rows[row] * dout[token]).sum(1)
    dx = torch.zeros_like(dout).index_add_(0, token, s["dgathered"].double()[row])
    return drows, dweights, dx


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "recur":
        return _exact_walk(s, _exact_decay(s), case["batch"])
    if case["op"] == "train":
        return _exact_train(s, case["batch"])
    return _exact_experts(s)
