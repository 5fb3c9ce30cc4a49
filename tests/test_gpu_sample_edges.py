"""sample_tokens at its edges: rows that are settled before their cuts, u at and past 1, and
rows so long that the bins' rounding grows."""
import numpy as np
import pytest
import torch

import prefix_scan_stream_amd as ps
from gpu_util import DEV, to_host
from test_gpu_sample import DTYPES, check, rows_of, uniforms, vec

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [900, 20000, 131072])
def test_rows_that_are_settled_early(vocab, dtype):
    """Greedy rows and rows with nothing left end in one wave, the others of their block with them;
    beside rows with cuts, and the same bits each time."""
    rows = 32
    x = rows_of(rows, vocab, DTYPES[dtype], vocab + 3)
    x[1::4] = -float("inf")
    t = np.where(np.arange(rows) % 4 == 2, 0.0, 0.8)
    u = uniforms(rows, 12)
    for cuts in (dict(k=np.full(rows, 20)), dict(p=np.full(rows, 0.9)), dict(k=np.full(rows, vocab // 2), p=np.full(rows, 0.8))):
        check(x, u, t, **cuts)
        args = vec(u), vec(t), vec(cuts.get("k"), torch.int32), vec(cuts.get("p"))
        first = [to_host(v) for v in ps.sample_tokens(x, *args)]
        for _ in range(20):
            again = ps.sample_tokens(x, *args)
        assert all((a == to_host(b)).all() for a, b in zip(first, again))
