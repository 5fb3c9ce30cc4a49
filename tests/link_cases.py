"""Cases of the gated recurrence whose values reach across tiles, groups of tiles and stretches, and a model of how
tiles are linked, whole or broken, in 64 bits.  The model has its own code; the kernels' layout is what it copies: tiles
of 64 or 128 tokens, eight tiles a group, and a stretch of one group or of eight."""
import numpy as np
import torch


TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
GATINGS = ["decay", "log", "sigmoid"]
# channels of one or two chains (links of groups and stretches of groups), and of six or more (of groups alone)
FEW = {"f32": 70, "f16": 67, "bf16": 70}
MANY = {"f32": 350, "f16": 643, "bf16": 642}


def rng(seed):
    return np.random.default_rng(20261209 + seed)


def slow_gates(r, shape, gating, dtype):
    """Gates of which some e^-2 is left after 8192 tokens."""
    if gating == "log":
        v = -2.5e-4 * (0.5 + r.random(shape))
    elif gating == "sigmoid":
        v = 8.3 + 0.2 * r.standard_normal(shape)
    else:
        # the type's largest value below 1 so often, and now and then a change of sign
        step = 2.0**-12 if dtype == torch.float32 else torch.finfo(dtype).eps / 2
        v = np.where(r.random(shape) < 2.0**-12 / step, 1 - step, 1.0) * np.where(r.random(shape) < 1 / 2000, -1, 1)
    return torch.from_numpy(v).to(dtype)


def slow_case(seed, shape, gating, dtype, sequences=1):
    """x, gate, dout, state and dstate_out whose sums grow: each channel's values have one sign."""
    r = rng(seed)
    sign = np.where(r.random(shape[-1]) < 0.5, -1.0, 1.0)
    size = 1.0 if gating == "sigmoid" else 2.0**-6
    some = lambda s: torch.from_numpy(s * sign * (0.5 + r.random(shape))).to(dtype)
    states = lambda: torch.from_numpy(sign * r.integers(3, 9, (sequences, shape[-1]))).float()
    return some(size), slow_gates(r, shape, gating, dtype), some(2.0**-6), states(), states()


def exact_case(seed, shape, dtype, sequences=1):
    """Decays of 1 and -1, and inputs of -1, 0 and 1: every product and sum is a small integer, which float32 holds."""
    r = rng(seed)
    some = lambda: torch.from_numpy(r.integers(-1, 2, shape).astype(np.float64)).to(dtype)
    states = lambda: torch.from_numpy(r.integers(3, 9, (sequences, shape[-1])) * np.where(r.random(shape[-1]) < 0.5, -1.0, 1.0)).float()
    return some(), torch.from_numpy(np.where(r.random(shape) < 0.02, -1.0, 1.0)).to(dtype), some(), states(), states()


def linked(a, b, first, tile, levels, broken=None):
    """h_t = a_t h_{t-1} + b_t of tokens x channels by tiles, groups and stretches; `broken` is one of BROKEN."""
    length, channels = a.shape
    tiles = -(-length // tile)
    pad = tiles * tile - length
    a = np.concatenate([a, np.ones((pad, channels))]).reshape(tiles, tile, channels)
    b = np.concatenate([b, np.zeros((pad, channels))]).reshape(tiles, tile, channels)
    factor, value = np.empty_like(a), np.empty_like(b)  # of the tile's first tokens
    f, v = np.ones((tiles, channels)), np.zeros((tiles, channels))
    for i in range(tile):
        f, v = f * a[:, i], v * a[:, i] + b[:, i]
        factor[:, i], value[:, i] = f, v
    maps = list(zip(factor[:, -1], value[:, -1]))
    if broken == "a tile's factor is lost":
        maps = [(0 * f, v) for f, v in maps]
    if broken == "a tile's factor is 1":
        maps = [(0 * f + 1, v) for f, v in maps]

    def compose(parts):
        f, v = np.ones(channels), np.zeros(channels)
        for of, ov in parts:
            f, v = f * of, of * v + ov
        if broken == "the last factor alone" and parts:
            f = parts[-1][0]
        if broken == "the maps in front are left out but the last" and parts:
            f, v = parts[-1]
        return f, v

    stretch = 8**levels
    front, h = first, np.empty_like(a)
    for p in range(tiles):
        group, start = p // 8 * 8, p // stretch * stretch
        near = compose(maps[group:p])
        far = compose([compose(maps[g:g + 8]) for g in range(start, group, 8)])
        if broken == "a group's factor is lost" and group > start:
            far = (0 * far[0], far[1])
        if broken == "groups in front are left out":
            far = (np.ones(channels), np.zeros(channels))
        shown = front
        if broken == "no front but for a group's first" and p > group:
            shown = 0 * front
        if broken == "no front but for a stretch's first" and p > start:
            shown = 0 * front
        if broken == "a stretch starts from zero" and start > 0:
            shown = 0 * front
        enters = near[0] * (far[0] * shown + far[1]) + near[1]
        h[p] = factor[p] * enters + value[p]
        if p == start + stretch - 1:
            front = maps[p][0] * enters + maps[p][1]
    return h.reshape(-1, channels)[:length]


BROKEN = {
    1: ["a tile's factor is lost", "a tile's factor is 1", "the last factor alone", "the maps in front are left out but the last",
        "no front but for a group's first", "a stretch starts from zero"],
    2: ["a tile's factor is lost", "a tile's factor is 1", "the last factor alone", "the maps in front are left out but the last",
        "no front but for a group's first", "no front but for a stretch's first", "a stretch starts from zero",
        "a group's factor is lost", "groups in front are left out"],
}


def room(dtype, want, bound):
    """How far an output of this type may be off: the bound before its rounding, half a step of that, and what is
    lost below float32's smallest normal value."""
    if dtype == torch.float32:
        return bound + 1e-37
    f = torch.finfo(dtype)
    return bound * (1 + f.eps / 2) + np.abs(want) * (f.eps / 2) + f.smallest_normal * f.eps + 1e-37
