"""Where sequences begin and end in a tile of packed rows: the kernels' own code (csrc/ls_marks.hpp), run on the CPU
with every index checked, against a loop over the sequences."""
import os
import subprocess

import numpy as np
import pytest

from prefix_scan_stream_amd import build as b

HERE = os.path.dirname(os.path.abspath(__file__))
TILE = 128


@pytest.fixture(scope="module")
def model(tmp_path_factory):
    exe = tmp_path_factory.mktemp("marks") / "row_marks_model"
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-I", b.CSRC, os.path.join(HERE, "row_marks_model.cpp"), "-o", str(exe)])

    def run(offsets, row0, rows=TILE, threads=512):
        offsets = np.asarray(offsets, dtype=np.int64)
        out = subprocess.run([str(exe), str(len(offsets) - 1), str(row0), str(rows), str(threads)], input=offsets.tobytes(),
                             stdout=subprocess.PIPE, timeout=60)
        assert out.returncode == 0, out.stdout.decode()
        reads, *lines = out.stdout.decode().split("\n")
        return int(reads), {int(l.split()[0]): tuple(map(int, l.split()[1:])) for l in lines if l}

    return run


def plain(offsets, row0, rows):
    marks = {}
    for s, (a, z) in enumerate(zip(offsets[:-1].tolist(), offsets[1:].tolist())):
        if z > a:
            if row0 <= a < row0 + rows:
                marks[a - row0] = (s, marks.get(a - row0, (-1, -1))[1])
            if row0 < z <= row0 + rows:
                marks[z - 1 - row0] = (marks.get(z - 1 - row0, (-1, -1))[0], s)
    return marks


def offsets_of(lengths):
    return np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)


LENGTHS = {
    "none": lambda r: [],
    "one": lambda r: [1000],
    "few": lambda r: r.integers(0, 200, 12),
    "empty ones among": lambda r: r.integers(0, 40, 500) * (r.random(500) < 0.2),
    "as many as threads": lambda r: r.integers(0, 4, 512),
    "one more than threads": lambda r: r.integers(0, 4, 513),
    "ones": lambda r: [1] * 3000,
    "mostly empty": lambda r: r.integers(1, 9, 60000) * (r.random(60000) < 0.01),
    "runs of empty ones": lambda r: np.concatenate([np.concatenate([np.zeros(n, int), [3]]) for n in
                                                    [5, 63, 64, 65, 511, 512, 513, 8191, 8192, 8193, 8255, 8256, 20000, 1, 0, 8703, 8704]]),
    "only empty ones": lambda r: [0] * 70000,
    "empty ones at the end": lambda r: [300] + [0] * 50000,
}


@pytest.mark.parametrize("threads", [64, 256, 512])
@pytest.mark.parametrize("name", LENGTHS)
def test_marks(model, name, threads):
    offsets = offsets_of(LENGTHS[name](np.random.default_rng(7)))
    end = int(offsets[-1])
    for row0 in sorted({0, 128, 256, end // 2 // 128 * 128, max(end - 1, 0) // 128 * 128, end // 128 * 128 + 128}):
        assert model(offsets, row0, threads=threads)[1] == plain(offsets, row0, TILE), (name, row0)


@pytest.mark.parametrize("count", [1 << 14, 1 << 18, 1 << 21])
@pytest.mark.parametrize("where", ["in front", "between", "behind"])
def test_empty_sequences_in_any_number_take_few_steps(model, count, where):
    """A tile's wait lasts a second at most, so no number of empty sequences at one row may hold it up: 16 rounds of
    the block's threads, a search of 64 probes a round, and some more rounds behind it."""
    empty = np.zeros(count, np.int64)
    lengths = {"in front": [empty, [50, 60]], "between": [[50], empty, [60]], "behind": [[50, 60], empty]}[where]
    offsets = offsets_of(np.concatenate(lengths))
    reads, marks = model(offsets, 0)
    assert marks == plain(offsets, 0, TILE)
    assert reads <= 200


@pytest.mark.parametrize("threads", [64, 512])
@pytest.mark.parametrize("seed", range(12))
def test_offsets_that_break_the_rules(model, seed, threads):
    """Out of order, negative, past the rows, at the ends of 64 bits: marks may be wrong, but no read leaves the
    offsets, no mark the tile, and every loop ends (the model checks all three)."""
    r = np.random.default_rng(seed)
    n = int(r.choice([1, 3, 100, 511, 512, 513, 2000, 30000]))
    wild = np.array([-(1 << 63), (1 << 63) - 1, -1, 0, 1, 127, 128, 129, 1 << 31, 1 << 40, -5])
    offsets = r.integers(-50, 400, n + 1)
    if seed % 3 == 0:
        offsets = np.sort(offsets)[::-1].copy()
    elif seed % 3 == 1:
        offsets = np.where(r.random(n + 1) < 0.3, r.choice(wild, n + 1), offsets)
    for row0 in (-128, 0, 128, 1 << 31):
        _, marks = model(offsets, row0, threads=threads)
        for row, (head, end) in marks.items():
            assert 0 <= row < TILE and -1 <= head < n and -1 <= end < n
