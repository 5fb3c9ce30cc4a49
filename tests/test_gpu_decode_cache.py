"""examples/decode_loop.py: what the model reads from the cache through the block table is
what the steps wrote for that request, and nothing else's."""
import pytest
import torch

from gpu_util import DEV
from test_gpu_decode_example import loop  # noqa: F401 - a fixture

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("requests,page,pages", [(1, 16, None), (64, 16, None), (300, 1, None), (300, 16, 700)])
def test_cached_keys_are_the_requests_own(loop, requests, page, pages):  # noqa: F811
    width, steps, bad = 64, [], []
    running = torch.zeros(requests, width, device=DEV)

    def on_step(owner, x, sums, done):
        # keys are whole numbers, so that sums in any order are the same
        live = owner >= 0
        running.index_add_(0, owner[live].long(), x[live])
        steps.append(int(live.sum()))
        if not torch.equal(sums, running) or bool(x[~live].any()):
            bad.append(len(steps))
        running.masked_fill_(done[:, None], 0.0)

    loop.serve(requests, 30, page, width=width, pages=pages, on_step=on_step)
    assert len(steps) == 30 and max(steps) > 0 and not bad
