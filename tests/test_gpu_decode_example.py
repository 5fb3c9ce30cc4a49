"""examples/decode_loop.py: the operators of a decoding step together, over many steps."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_loop.py")


@pytest.fixture(scope="module")
def loop():
    spec = importlib.util.spec_from_file_location("decode_loop", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("requests,page,pages", [(1, 16, None), (64, 16, None), (300, 1, None), (300, 16, 700)])
def test_pages_are_neither_lost_nor_shared(loop, requests, page, pages):
    """After many steps every page is in one table or on the free list, once, also when the
    pool is too small for all requests; each request holds the pages of its length."""
    tokens, lens, tables, free, count, generated = loop.serve(requests, 30, page, pages=pages)
    n = int(count)
    held = tables[tables >= 0]
    everything = torch.cat([held, free[:n]]).sort().values
    assert torch.equal(everything, torch.arange(free.numel(), dtype=torch.int32, device=free.device))
    want = (lens + page - 1) // page
    assert torch.equal((tables >= 0).sum(1).int(), want)
    assert bool(((tokens >= 0) & (tokens < 4096)).all())
    if pages is None:
        assert int(generated.sum()) > 0
    else:
        assert 0 < int(generated.sum()) < 30 * requests


def test_same_tokens_every_time(loop):
    first, again = loop.serve(64, 12), loop.serve(64, 12)
    assert torch.equal(first[5], again[5]) and torch.equal(first[1], again[1])
