"""That the cases which test the linking of tiles on the GPU see a link that is broken (CPU only): the linked model gives
the oracle's values, and each way to break it is off by more than the tests allow, forward and backward."""
import numpy as np
import pytest
import torch

import layer_oracle as lo
import link_cases as lc

LENGTHS = {1: 2700, 2: 8192 + 1500}


def host(t):
    return t.double().numpy()


def sides(x, gate, dout, state, dstate, gating):
    """Forward and backward as h = a h + b of tokens x channels: (factors, summands, first value, wanted, bound, shown),
    where shown() makes the tested output of the recurrence's values."""
    x, gate, dout, state, dstate = (host(t) for t in (x, gate, dout, state, dstate))
    a, _ = lo.decay(gate, gating)
    rest = lo.rest_of(gate) if gating == "sigmoid" else np.ones_like(a)
    h, hb, _ = lo.recurrence(x[None], gate[None], state[None], gating)
    (dx, _, _), (ex, _, _) = lo.gradients(x[None], gate[None], state[None], dout[None], dstate[None], gating)

    def backward(mu):  # mu[t]: what leaves token t towards the first, last token first
        lam = dout[::-1] + np.concatenate([dstate[None], mu[:-1]])
        return (lam * rest[::-1])[::-1]

    return {"forward": (a, rest * x, state, h[0], hb[0], lambda v: v),
            "backward": (a[::-1], (a * dout)[::-1], dstate, dx[0], ex[0], backward)}


@pytest.mark.parametrize("dtype", lc.TYPES)
@pytest.mark.parametrize("gating", lc.GATINGS + ["exact"])
@pytest.mark.parametrize("levels", [1, 2])
def test_broken_links_are_seen(levels, gating, dtype):
    t, few = lc.TYPES[dtype], 4
    shape = (LENGTHS[levels], (lc.MANY if levels == 1 else lc.FEW)[dtype])
    if gating == "exact":
        case, gating = lc.exact_case(levels, shape, t), "decay"
    else:
        case = lc.slow_case(levels, shape, gating, t)
    x, gate, dout, (state,), (dstate,) = (v[:, :few] for v in case)
    case = x, gate, dout, state, dstate
    for side, (a, b, first, want, bound, shown) in sides(*case, gating).items():
        allowed = lc.room(t, want, bound)
        for tile in (64, 128) if side == "backward" else (128,):
            whole = shown(lc.linked(a, b, first, tile, levels))
            assert (np.abs(whole - want) <= bound).all(), side
            for broken in lc.BROKEN[levels]:
                wrong = np.abs(shown(lc.linked(a, b, first, tile, levels, broken)) - want)
                # not by a hair, and in every channel
                assert (np.max(wrong / allowed, axis=0) > 2).all(), (side, tile, broken)


def test_exact_cases_are_exact():
    """Values and products of the integer cases stay below 2^24, in the longest of them."""
    for seed in (1, 2):
        x, gate, dout, state, dstate = lc.exact_case(seed, (20000, 60), torch.float32)
        h, _, last = lo.recurrence(host(x)[None], host(gate)[None], host(state), "decay")
        (dx, dg, ds), _ = lo.gradients(host(x)[None], host(gate)[None], host(state), host(dout)[None], host(dstate), "decay")
        for v in (h, last, dx, dg, ds):
            assert (np.abs(v) < 2**24).all() and (v == np.rint(v)).all()
