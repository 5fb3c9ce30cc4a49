"""The operators of a decoding step, as measured cases.

sample       a batch of logit rows to one token each (ps.sample_tokens)
append       pages for the tokens of this step, taken from the free list (ps.pages_append)
slots        cache slots, positions and request numbers of this step's tokens (ps.slot_map)
release      the pages of finished requests back on the free list (ps.pages_release)

A case is a dict of plain values; listed() and draw() make them, prepare() makes the
tensors a serving program holds before the call, run() is the call itself: in elementary
torch operations where `own` is false, with the library where it is true.
"""
import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one chat: a single row, all cuts in force; latency is what counts
        dict(name="sample-1", op="sample", rows=1, vocab=131072, pad=0, dtype="bfloat16", spread=2.5, temperature=0.8,
             greedy=0.0, top_k=50, top_p=0.95, min_p=0.02, masked=0.0),
        # a small batch of constrained requests: an odd vocabulary in a padded buffer, most tokens
        # masked by a grammar, some rows greedy, one in eight with nothing left
        dict(name="sample-13-masked", op="sample", rows=13, vocab=50003, pad=61, dtype="float16", spread=3.0,
             temperature=1.0, greedy=0.3, top_k=40, top_p=0.9, min_p=0.0, masked=0.7),
        # a serving batch with the usual cuts
        dict(name="sample-64", op="sample", rows=64, vocab=131072, pad=0, dtype="bfloat16", spread=2.5,
             temperature=0.7, greedy=0.0, top_k=100, top_p=0.9, min_p=0.05, masked=0.0),
        # a large batch cut by mass alone
        dict(name="sample-256-nucleus", op="sample", rows=256, vocab=131072, pad=0, dtype="bfloat16", spread=2.0,
             temperature=1.0, greedy=0.0, top_k=0, top_p=0.95, min_p=0.0, masked=0.0),
        # rollouts for training: the whole distribution, float32 logits
        dict(name="sample-512-full", op="sample", rows=512, vocab=131072, pad=0, dtype="float32", spread=2.0,
             temperature=1.0, greedy=0.0, top_k=0, top_p=1.0, min_p=0.0, masked=0.0),
        # one decoding step of a full batch: a token each, a new page now and then
        dict(name="append-decode-256", op="append", requests=256, page=16, longest=8192, new=1, columns=544,
             scarce=False),
        # a wave of long prompts that the free list just does not hold
        dict(name="append-prefill-4096", op="append", requests=4096, page=16, longest=64, new=32768, columns=2056,
             scarce=True),
        # the decoding step's slots
        dict(name="slots-decode-256", op="slots", requests=256, page=16, longest=8192, new=1, columns=544, extra=0),
        # prompts in chunks among decoding requests, odd page size, a buffer of fixed length
        dict(name="slots-mixed-700", op="slots", requests=700, page=24, longest=4096, new=90, columns=180, extra=1000),
        # a wave of prompts
        dict(name="slots-prefill-1024", op="slots", requests=1024, page=64, longest=512, new=8192, columns=140,
             extra=0),
        # a tenth of a batch has finished
        dict(name="release-512", op="release", requests=512, page=16, longest=8192, columns=520, finished=0.1),
        # a cache is emptied
        dict(name="release-4096", op="release", requests=4096, page=16, longest=32768, columns=2056, finished=0.98),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["sample", "sample", "sample", "append", "slots", "release"])
    if op == "sample":
        vocab = _log_int(rng, 1000, 131072)
        rows = _log_int(rng, 1, max(1, min(512, (1 << 25) // vocab)))
        return dict(op=op, rows=rows, vocab=vocab, pad=rng.choice([0, 0, 1, 8, rng.randint(0, 200)]),
                    dtype=rng.choice(["float32", "float16", "bfloat16"]), spread=rng.uniform(0.5, 4.0),
                    temperature=rng.choice([1.0, rng.uniform(0.3, 1.5)]), greedy=rng.choice([0.0, 0.0, 0.25]),
                    top_k=rng.choice([0, 0, 1, rng.randint(2, 64), _log_int(rng, 64, vocab)]),
                    top_p=rng.choice([1.0, 1.0, rng.uniform(0.5, 0.99), rng.uniform(0.05, 0.5)]),
                    min_p=rng.choice([0.0, 0.0, rng.uniform(0.001, 0.2)]),
                    masked=rng.choice([0.0, 0.0, rng.uniform(0.1, 0.95)]))
    page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
    requests = _log_int(rng, 1, 4096)
    if op == "release":
        longest = _log_int(rng, 16, 4096)
        return dict(op=op, requests=requests, page=page, longest=longest, columns=-(-longest // page) + rng.randint(0, 9),
                    finished=rng.choice([0.05, 0.5, 1.0]))
    new = rng.choice([1, _log_int(rng, 2, 1024)])
    longest = _log_int(rng, 16, 2048)
    case = dict(op=op, requests=requests, page=page, longest=longest, new=new,
                columns=-(-(longest + new) // page) + rng.randint(0, 9))
    if op == "append":
        case["scarce"] = rng.random() < 0.3
    else:
        case["extra"] = rng.choice([0, 0, 7, 500])
    return case


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _sample_inputs(case, seed):
    g = _generator(seed)
    rows, vocab = case["rows"], case["vocab"]
    full = torch.empty(rows, vocab + case["pad"], device=DEV, dtype=DTYPES[case["dtype"]])
    for r0 in range(0, rows, 64):
        part = full[r0:r0 + 64]
        x = torch.randn(part.shape, device=DEV, generator=g) * case["spread"]
        # a few tokens stand out, as a trained model's do
        hot = torch.rand(part.shape, device=DEV, generator=g) < 20.0 / vocab
        lift = -torch.log(torch.rand(part.shape, device=DEV, generator=g).clamp_min(1e-7)) * 3.0 + 4.0
        x = torch.where(hot, x + lift, x)
        if case["masked"] > 0:
            drop = torch.rand(part.shape, device=DEV, generator=g) < case["masked"]
            x = x.masked_fill(drop, float("-inf"))
        part.copy_(x)
    if case["masked"] > 0:
        full[3::8] = float("-inf")  # nothing left
        full[5::8, : vocab // 2] = torch.finfo(full.dtype).min  # masked by the type's lowest value
    per_row = lambda low, high: torch.rand(rows, device=DEV, generator=g) * (high - low) + low
    temperature = per_row(0.9, 1.1) * case["temperature"]
    if case["greedy"] > 0:
        temperature[torch.rand(rows, device=DEV, generator=g) < case["greedy"]] = 0.0
    state = dict(logits=full[:, :vocab], uniforms=torch.rand(rows, device=DEV, generator=g), temperature=temperature,
                 top_k=None, top_p=None, min_p=None)
    if case["top_k"] > 0:
        state["top_k"] = (case["top_k"] * per_row(0.8, 1.0)).ceil().to(torch.int32)
    if case["top_p"] < 1:
        state["top_p"] = case["top_p"] * per_row(0.97, 1.0)
    if case["min_p"] > 0:
        state["min_p"] = case["min_p"] * per_row(0.8, 1.2)
    return state


def _mean_new(case):
    """Tokens a request adds in this step, on average."""
    return 0 if case["op"] == "release" else 1 if case["new"] == 1 else 0.25 + 0.7 * (case["new"] + 1) / 2


def _budget(case):
    return max(1, int(case["requests"] * _mean_new(case) * (1 if case["new"] == 1 else 0.9)))


def _cache_inputs(case, seed):
    """Lengths, a block table whose used part holds a random permutation's pages, and the
    rest of the pool's pages on the free list."""
    g = _generator(seed)
    rows, page, columns = case["requests"], case["page"], case["columns"]
    lens = torch.randint(1, case["longest"] + 1, (rows,), device=DEV, generator=g)
    if case["op"] == "release":
        new = torch.zeros_like(lens)
    elif case["new"] == 1:
        new = torch.ones_like(lens)
    else:
        # prompts of very different lengths, some requests only decoding, a few idle
        new = torch.randint(1, case["new"] + 1, (rows,), device=DEV, generator=g)
        kind = torch.rand(rows, device=DEV, generator=g)
        new = torch.where(kind < 0.25, torch.ones_like(new), new)
        new = torch.where(kind > 0.95, torch.zeros_like(new), new)
    if case["op"] == "slots":
        # the scheduler stops at its budget of tokens for a step
        new = (_budget(case) - (torch.cumsum(new, 0) - new)).clamp_min(0).minimum(new)
    have = (lens + page - 1) // page
    want = (lens + new + page - 1) // page
    held = want if case["op"] == "slots" else have
    used, asked = int(held.sum()), int((want - have).sum())
    # the pool: what tables of uniform lengths need and some more
    pages = rows * columns if rows < 64 else rows * columns * 5 // 8
    order = torch.randperm(pages, device=DEV, generator=g).to(torch.int32)
    first = torch.cumsum(held, 0) - held
    col = torch.arange(columns, device=DEV)
    at = (first[:, None] + col).clamp_max(pages - 1)
    tables = torch.where(col < held[:, None], order[at], torch.full((), -1, device=DEV, dtype=torch.int32))
    free = torch.full((pages,), -1, device=DEV, dtype=torch.int32)
    free[: pages - used] = order[used:]
    count = pages - used
    if case.get("scarce"):
        count = asked * 15 // 16
    state = dict(lens=lens.to(torch.int32), new_lens=new.to(torch.int32), tables=tables.contiguous(), free_pages=free,
                 free_count=torch.tensor([count], device=DEV), page_size=page)
    if case["op"] == "slots":
        state["capacity"] = _budget(case) + case["extra"]
    if case["op"] == "release":
        state["finished"] = torch.rand(rows, device=DEV, generator=g) < case["finished"]
    return state


def prepare(case, seed):
    state = _sample_inputs(case, seed) if case["op"] == "sample" else _cache_inputs(case, seed)
    state["op"] = case["op"]
    if own:
        import prefix_scan_stream_amd as ps
        ps.load_library()
        # the buffers that a serving program keeps from step to step
        if case["op"] == "sample":
            rows = case["rows"]
            state["out"] = torch.empty(rows, device=DEV, dtype=torch.int64)
            state["logprobs"] = torch.empty(rows, device=DEV)
        else:
            state["count_out"] = torch.empty(1, device=DEV, dtype=torch.int64)
            state["granted"] = torch.empty(case["requests"], device=DEV, dtype=torch.bool)
            if case["op"] == "slots":
                n = state["capacity"]
                state["out"] = (torch.empty(n, device=DEV, dtype=torch.int64), torch.empty(n, device=DEV, dtype=torch.int32),
                                torch.empty(n, device=DEV, dtype=torch.int32),
                                torch.empty(case["requests"] + 1, device=DEV, dtype=torch.int64))
    return state


# ------------------------------------------------------------------ plain forms

def _plain_sample(s):
    # adding zero makes -0 and 0 one value; what is not a number counts as masked
    x = s["logits"].to(torch.float64) + 0.0
    x = torch.where(torch.isnan(x), torch.full_like(x, float("-inf")), x)
    top = x.amax(1, keepdim=True)
    best = x.argmax(1)
    t = s["temperature"].to(torch.float64)[:, None]
    # the prefix sums decide between neighbouring tokens, so all of this is in 64 bits
    d = torch.where(x == top, torch.zeros_like(x), (top - x) / t)
    d = torch.where(x == float("-inf"), torch.full_like(x, float("inf")), d)
    w = torch.exp(-d)
    kept = w
    if s["top_k"] is not None or s["top_p"] is not None:
        order = torch.sort(x, dim=1, descending=True, stable=True).indices
        ws = torch.gather(w, 1, order)
        rank = torch.arange(x.shape[1], device=x.device)
        if s["top_k"] is not None:
            ws = torch.where(rank < s["top_k"][:, None], ws, torch.zeros_like(ws))
        if s["top_p"] is not None:
            running = torch.cumsum(ws, 1)
            before = torch.cat([torch.zeros_like(running[:, :1]), running[:, :-1]], 1)
            goal = s["top_p"].to(torch.float64)[:, None] * running[:, -1:]
            ws = torch.where((before < goal) | (rank == 0), ws, torch.zeros_like(ws))
        kept = torch.zeros_like(w).scatter_(1, order, ws)
    if s["min_p"] is not None:
        kept = torch.where(w >= s["min_p"].to(torch.float64).clamp_max(1.0)[:, None], kept, torch.zeros_like(kept))
    running = torch.cumsum(kept, 1)
    total = running[:, -1]
    goal = s["uniforms"].to(torch.float64) * total
    token = (running > goal[:, None]).to(torch.uint8).argmax(1)
    logprob = -torch.gather(d, 1, token[:, None])[:, 0] - torch.log(total)
    greedy = s["temperature"] <= 0
    token = torch.where(greedy, best, token)
    logprob = torch.where(greedy, torch.zeros_like(logprob), logprob)
    empty = top[:, 0] == float("-inf")
    token = torch.where(empty, torch.full_like(token, -1), token)
    logprob = torch.where(empty, torch.full_like(logprob, float("-inf")), logprob)
    return token, logprob.to(torch.float32)


def _plain_append(s):
    page, tables, free = s["page_size"], s["tables"], s["free_pages"]
    columns = tables.shape[1]
    lens, new = s["lens"].long(), s["new_lens"].long()
    have = (lens + page - 1) // page
    want = (lens + new + page - 1) // page
    fits = want <= columns
    need = torch.where(fits, want - have, torch.zeros_like(want))
    upto = torch.cumsum(need, 0)
    count = s["free_count"][0]
    granted = fits & ((need == 0) | (upto <= count))
    taken = torch.where(upto <= count, upto, torch.zeros_like(upto)).max()
    col = torch.arange(columns, device=tables.device)
    at = count - 1 - ((upto - need - have)[:, None] + col)
    fresh = granted[:, None] & (col >= have[:, None]) & (col < want[:, None])
    tables = torch.where(fresh, free[at.clamp(0, free.numel() - 1)], tables)
    return tables, granted, (count - taken).reshape(1)


def _plain_slots(s):
    page, tables, n = s["page_size"], s["tables"], s["capacity"]
    lens, new = s["lens"].long(), s["new_lens"].long()
    ends = torch.cumsum(new, 0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    t = torch.arange(n, device=tables.device)
    r = torch.searchsorted(ends, t, right=True)
    live = r < lens.numel()
    r = r.clamp_max(lens.numel() - 1)
    at = lens[r] + t - offsets[r]
    col = at // page
    held = torch.where(col < tables.shape[1], tables[r, col.clamp_max(tables.shape[1] - 1)].long(), torch.full_like(col, -1))
    slots = torch.where(live & (held >= 0), held * page + at % page, torch.full_like(at, -1))
    positions = torch.where(live, at, torch.zeros_like(at)).to(torch.int32)
    requests = torch.where(live, r, torch.full_like(r, -1)).to(torch.int32)
    return slots, positions, requests, offsets


def _plain_release(s):
    page, tables, free = s["page_size"], s["tables"], s["free_pages"]
    columns = tables.shape[1]
    held = ((s["lens"].long() + page - 1) // page).clamp_max(columns)
    held = torch.where(s["finished"], held, torch.zeros_like(held))
    upto = torch.cumsum(held, 0)
    count = s["free_count"][0]
    i = torch.arange(free.numel(), device=tables.device) - count
    r = torch.searchsorted(upto, i, right=True)
    back = (i >= 0) & (r < held.numel())
    r = r.clamp_max(held.numel() - 1)
    col = (i - (upto - held)[r]).clamp(0, columns - 1)
    return torch.where(back, tables[r, col], free), (count + upto[-1]).reshape(1)


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["op"]
    if not own:
        return {"sample": _plain_sample, "append": _plain_append, "slots": _plain_slots, "release": _plain_release}[op](state)
    import prefix_scan_stream_amd as ps
    if op == "sample":
        return ps.sample_tokens(state["logits"], state["uniforms"], temperature=state["temperature"],
                                top_k=state["top_k"], top_p=state["top_p"], min_p=state["min_p"], out=state["out"],
                                logprobs=state["logprobs"])
    if op == "append":
        count, granted = ps.pages_append(state["lens"], state["new_lens"], state["tables"], state["free_pages"],
                                         state["free_count"], state["page_size"], count_out=state["count_out"],
                                         granted=state["granted"])
        return state["tables"], granted, count
    if op == "slots":
        return ps.slot_map(state["lens"], state["new_lens"], state["tables"], state["page_size"], state["capacity"],
                           out=state["out"])
    count = ps.pages_release(state["lens"], state["finished"], state["tables"], state["free_pages"], state["free_count"],
                             state["page_size"], count_out=state["count_out"])
    return state["free_pages"], count


def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        size = 4 if case["dtype"] == "float32" else 2
        cuts = sum((case["top_k"] > 0, case["top_p"] < 1, case["min_p"] > 0))
        # a difference, a scaling, an exponential and a sum for each logit
        return {"bytes": n * size + case["rows"] * (4 + 4 + 4 * cuts + 12), "flops": 4 * n}
    rows, page = case["requests"], case["page"]
    mean_new = _mean_new(case)
    if case["op"] == "append":
        pages = rows * mean_new / page * (15 / 16 if case["scarce"] else 1)
        return {"bytes": int(rows * 9 + pages * 8 + 16), "flops": int(rows * 8)}
    if case["op"] == "slots":
        tokens = _budget(case)
        return {"bytes": int(rows * 16 + 8 + tokens * 16 + case["extra"] * 16 + (tokens / page + rows / 2) * 4),
                "flops": int(tokens * 4)}
    pages = rows * case["finished"] * (case["longest"] / 2 / page + 0.5)
    return {"bytes": int(rows * 5 + pages * 8 + 16), "flops": int(rows * 4)}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_sample(s):
    tokens, logprobs = [], []
    rows, vocab = s["logits"].shape
    for r in range(rows):
        x = s["logits"][r].double()
        x[x != x] = float("-inf")
        t = float(s["temperature"][r])
        top = float(x.max())
        if top == float("-inf"):
            tokens.append(-1)
            logprobs.append(float("-inf"))
            continue
        if t <= 0:
            tokens.append(int(torch.nonzero(x == top)[0]))
            logprobs.append(0.0)
            continue
        w = torch.exp((x - top) / t)
        values, index = torch.sort(-x, stable=True)
        ordered = w[index]
        keep = vocab
        if s["top_k"] is not None:
            keep = min(keep, int(s["top_k"][r]))
        if s["top_p"] is not None:
            sums = torch.cumsum(ordered[:keep], 0)
            goal = float(s["top_p"][r]) * float(sums[-1])
            keep = min(keep, int((sums < goal).sum()) + 1)
        if s["min_p"] is not None:
            keep = min(keep, max(1, int((ordered >= min(1.0, float(s["min_p"][r]))).sum())))
        chosen, _ = torch.sort(index[:keep])
        sums = torch.cumsum(w[chosen], 0)
        total = float(sums[-1])
        at = int((sums <= float(s["uniforms"][r]) * total).sum())
        token = int(chosen[min(at, keep - 1)])
        tokens.append(token)
        logprobs.append((float(x[token]) - top) / t - math.log(total))
    return (torch.tensor(tokens, dtype=torch.int64, device=DEV),
            torch.tensor(logprobs, dtype=torch.float64, device=DEV))


def _exact_cache(s):
    op, page = s["op"], s["page_size"]
    lens, tables, free = s["lens"].tolist(), s["tables"].cpu().clone(), s["free_pages"].cpu().clone()
    count = int(s["free_count"])
    pages = lambda tokens: -(-tokens // page)
    if op == "release":
        for r, done in enumerate(s["finished"].tolist()):
            if done:
                n = min(pages(lens[r]), tables.shape[1])
                free[count:count + n] = tables[r, :n]
                count += n
        return free.to(DEV), torch.tensor([count], device=DEV)
    new = s["new_lens"].tolist()
    if op == "append":
        granted, stopped = [], False
        for r, length in enumerate(lens):
            have, want = pages(length), pages(length + new[r])
            n = want - have
            if want > tables.shape[1]:
                granted.append(False)
                continue
            stopped = stopped or n > count
            granted.append(n == 0 or not stopped)
            if n and not stopped:
                tables[r, have:want] = free[count - n:count].flip(0)
                count -= n
        return tables.to(DEV), torch.tensor(granted, device=DEV), torch.tensor([count], device=DEV)
    n, at = s["capacity"], 0
    slots = torch.full((n,), -1, dtype=torch.int64)
    positions, requests = torch.zeros(n, dtype=torch.int32), torch.full((n,), -1, dtype=torch.int32)
    offsets = [0]
    for r, length in enumerate(lens):
        where = torch.arange(length, length + new[r])
        slots[at:at + new[r]] = tables[r, where // page].long() * page + where % page
        positions[at:at + new[r]] = where.int()
        requests[at:at + new[r]] = r
        at += new[r]
        offsets.append(at)
    return slots.to(DEV), positions.to(DEV), requests.to(DEV), torch.tensor(offsets, device=DEV)


def exact(case, seed):
    state = prepare(case, seed)
    return _exact_sample(state) if case["op"] == "sample" else _exact_cache(state)
