"""The operators together, as a layer uses them: the recurrence over a step's packed rows (offsets and
rows from pages_append and slot_map), a router, the experts' products, and all gradients."""
import numpy as np
import pytest
import torch

import prefix_scan_stream_amd as ps

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Recurrence(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, state, offsets):
        carries = ps.recurrence_carries(x, offsets)
        out = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        out, last = ps.gated_recurrence(x, gate, state=state, offsets=offsets, out=out, carries=carries)
        ctx.save_for_backward(x, gate, state, offsets, carries)
        return out, last

    @staticmethod
    def backward(ctx, dout, dlast):
        x, gate, state, offsets, carries = ctx.saved_tensors
        dx, dgate = torch.zeros_like(x), torch.zeros_like(gate)
        dx, dgate, dstate = ps.gated_recurrence_backward(dout.contiguous(), x, gate, carries, state=state,
                                                         dstate_out=dlast.contiguous(), offsets=offsets, dx=dx, dgate=dgate)
        return dx, dgate, dstate, None


class Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, places):
        ctx.save_for_backward(places)
        return ps.experts_gather(x, places, out=torch.zeros(places.numel(), x.shape[1], dtype=x.dtype, device=x.device))

    @staticmethod
    def backward(ctx, drows):
        return ps.experts_combine(drows.contiguous(), *ctx.saved_tensors), None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, places):
        ctx.save_for_backward(rows, weights, places)
        return ps.experts_combine(rows, places, weights)

    @staticmethod
    def backward(ctx, dout):
        rows, weights, places = ctx.saved_tensors
        drows, dweights = ps.experts_combine_backward(dout.contiguous(), rows, places, weights, drows=torch.zeros_like(rows))
        return drows, dweights, None


def layer(w, x, state, lens, experts, sort, recurrence, dispatch, combine):
    """w: projection (d, 2d), router (d, E), experts (E, d, d).  experts: the choice, or None to make it."""
    proj = x @ w[0]
    d = x.shape[1]
    h, last = recurrence(proj[:, :d], proj[:, d:], state)
    scores = torch.softmax(h @ w[1], 1)
    if experts is None:
        experts = torch.topk(scores, 2, dim=1).indices
        live = torch.arange(x.shape[0], device=x.device)[:, None] < lens
        experts = torch.where(live, experts, torch.full_like(experts, -1))
    weights = torch.gather(scores, 1, experts.clamp_min(0))
    offsets, places = sort(experts)
    rows = dispatch(h, places)
    bounds = offsets.tolist()
    made = torch.cat([rows[a:b] @ w[2][e] for e, (a, b) in enumerate(zip(bounds[:-1], bounds[1:]))] + [rows[bounds[-1]:] * 0])
    return combine(made, weights, places) + h, last, experts


def test_layer_and_its_gradients():
    g = torch.Generator().manual_seed(4)
    rand = lambda *s: torch.randn(*s, generator=g)
    requests, d, num, page = 6, 48, 5, 16
    lens = torch.tensor([3, 0, 40, 7, 9, 1], dtype=torch.int32, device=DEV)
    new = torch.tensor([1, 90, 33, 0, 1, 1], dtype=torch.int32, device=DEV)
    tables = torch.full((requests, 8), -1, dtype=torch.int32, device=DEV)
    free, count = torch.arange(64, dtype=torch.int32, device=DEV), torch.tensor([64], device=DEV)
    ps.pages_append(torch.zeros_like(lens), lens, tables, free, count, page)
    capacity = 140
    _, _, owner, offsets = ps.slot_map(lens, new, tables, page, capacity)
    live = int(offsets[-1])
    assert live == 126 and int((owner >= 0).sum()) == live

    x = rand(capacity, d)
    w = [rand(d, 2 * d) / d**0.5, rand(d, num), rand(num, d, d) / d**0.5]
    state, up, uplast = rand(requests, d), rand(capacity, d), rand(requests, d)
    up[live:] = 0  # rows behind the last token have no loss

    leaves = [t.to(DEV).requires_grad_() for t in (x, *w, state)]
    out, last, experts = layer(
        leaves[1:4], leaves[0], leaves[4], live, None, lambda e: (lambda r: (r[0], r[2]))(ps.experts_sort(e, num)),
        lambda a, b, s: Recurrence.apply(a, b, s, offsets), Dispatch.apply, Combine.apply)
    loss = (out * up.to(DEV)).sum() + (last * uplast.to(DEV)).sum()
    got = torch.autograd.grad(loss, leaves)

    # the same in float64 on the CPU, from the definitions, with the same choice of experts
    bounds = offsets.tolist()

    def recurrence(a, b, s):
        rows, final = [], []
        for r in range(requests):
            h = s[r]
            for t in range(bounds[r], bounds[r + 1]):
                decay = torch.sigmoid(b[t])
                h = decay * h + (1 - decay) * a[t]
                rows.append(h)
            final.append(h)
        rows += [torch.zeros(d, dtype=torch.float64)] * (capacity - bounds[-1])
        return torch.stack(rows), torch.stack(final)

    def sort(e):
        flat = e.reshape(-1)
        order = torch.cat([torch.nonzero(flat == k)[:, 0] for k in range(num)])
        places = torch.full_like(flat, -1)
        places[order] = torch.arange(order.numel())
        sizes = torch.stack([(flat == k).sum() for k in range(num)])
        return torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]), places.reshape(e.shape)

    def dispatch(h, places):
        t, j = torch.nonzero(places >= 0, as_tuple=True)
        return torch.zeros(places.numel(), d, dtype=torch.float64).index_put((places[t, j],), h[t])

    def combine(rows, weights, places):
        return (rows[places.clamp_min(0)] * (weights * (places >= 0))[:, :, None]).sum(1)

    exact = [t.double().requires_grad_() for t in (x, *w, state)]
    eout, elast, _ = layer(exact[1:4], exact[0], exact[4], live, experts.cpu(), sort, recurrence, dispatch, combine)
    eloss = (eout * up.double()).sum() + (elast * uplast.double()).sum()
    want = torch.autograd.grad(eloss, exact)
    assert torch.allclose(out[:live].double().cpu(), eout[:live].detach(), rtol=0, atol=1e-4)
    assert torch.allclose(last.double().cpu(), elast.detach(), rtol=0, atol=1e-4)
    for a, b in zip(got, want):
        # float32 through five products of up to 96 terms and sums over 126 tokens: some 1e-6 relative each
        assert (a.double().cpu() - b).norm() <= 1e-4 * b.norm()


def test_a_step_continues_where_the_last_ended():
    """A prompt in pieces, the state handed on in place, then single tokens: h as of the whole sequence."""
    g = torch.Generator().manual_seed(8)
    x, gate = (torch.randn(300, 96, generator=g).to(DEV) for _ in range(2))
    whole, final = ps.gated_recurrence(x[None], gate[None])
    state = torch.zeros(1, 96, device=DEV)
    parts, at = [], 0
    for n in (130, 1, 100, 63, 1, 1, 1, 1, 1, 1):
        off = torch.tensor([0, n], device=DEV)
        if n > 1:
            h, _ = ps.gated_recurrence(x[at:at + n], gate[at:at + n], state=state, offsets=off, state_out=state)
        else:
            h, _ = ps.gated_recurrence(x[at:at + 1], gate[at:at + 1], state=state, state_out=state)
        parts.append(h)
        at += n
    assert at == 300
    # |h| < 6; each way rounds an h some 300 times at most, with decays below 1
    assert float((torch.cat(parts) - whole[0]).abs().max()) < 300 * 6 * 2.0**-24 * 12
    assert float((state - final).abs().max()) < 300 * 6 * 2.0**-24 * 12


def test_rows_that_no_place_names_in_deterministic_mode():
    """torch's deterministic mode fills new tensors, and the rows that the calls leave alone show it: the same on
    every run."""
    x = torch.randn(6, 40, device=DEV)
    places = torch.tensor([[0, 2], [1, -1], [-1, 3], [4, 5], [6, 7], [9, -1]], dtype=torch.int32, device=DEV)
    named = places[places >= 0].long()
    free = torch.ones(12, dtype=torch.bool, device=DEV)
    free[named] = False
    weights = torch.rand(6, 2, device=DEV)
    rows = torch.randn(12, 40, device=DEV)
    torch.use_deterministic_algorithms(True)
    try:
        got = ps.experts_gather(x, places)
        drows, _ = ps.experts_combine_backward(x, rows, places, weights)
    finally:
        torch.use_deterministic_algorithms(False)
    for t in (got, drows):
        assert bool(t[free].isnan().all()) and bool(torch.isfinite(t[named]).all())
    assert bool(torch.isfinite(ps.experts_combine(rows, places, weights)).all())
