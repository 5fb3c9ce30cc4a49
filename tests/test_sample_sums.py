"""How far the sums of sample_tokens' cuts by value may be off, by a model of the bins'
integers: the statement of libscan.h, for rows of every length."""
import math
import os
import re

import numpy as np
import pytest

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "libscan.h")


def stated(vocab):
    """The relative error of a row's sum that libscan.h allows a cut by value."""
    return 2.0 ** -min(44, 61 - math.ceil(math.log2(vocab)))


def off(vocab, log2w, per_octave):
    """The largest relative error of weights 2^-x as integers of 2^-frac of their bin's weight (per_octave 8)
    or of their octave's (1), with the weights that the bins leave out."""
    frac = min(44, 61 - math.ceil(math.log2(vocab)))
    unit = np.exp2(-np.rint(log2w * 8) // (8 // per_octave) / per_octave - frac)
    w = np.exp2(-log2w)
    left_out = vocab * 2.0**-63.9 if per_octave == 8 else 0.0
    return float((np.abs(np.rint(w / unit) * unit - w) / w).max()) + left_out + 2.0**-48.9


LENGTHS = [1000, 1 << 17, (1 << 17) + 1, 151936, 1 << 18, 262145, 1_200_007, 1 << 24, 1 << 28, 2**31 - 1]


@pytest.mark.parametrize("vocab", LENGTHS)
def test_the_statement_holds(vocab):
    log2w = np.random.default_rng(vocab).uniform(0, 60, 400_000)
    worst = max(off(vocab, log2w, 8), off(vocab, log2w, 1))
    assert worst <= stated(vocab)
    if vocab > 1 << 19:
        assert worst > 2.0**-44  # what rows of up to 2^17 keep to does not hold for these


def test_the_header_says_so():
    with open(HEADER) as f:
        text = " ".join(f.read().replace(" * ", " ").split())
    assert "2^-44 if vocab <= 2^17 or there are no cuts" in text
    assert "up to 2^-(61 - ceil(log2 vocab))" in text
    examples = re.findall(r"2\^-(\d+) for 2\^(\d+)", text)
    assert len(examples) == 3
    for bits, length in examples:
        assert stated(2 ** int(length)) == 2.0 ** -int(bits)
