"""A serving loop on the operators of a decoding step, with a toy model.

    python examples/decode_loop.py [--requests 64] [--steps 40] [--page-size 16]

Each step, for a batch of requests of different lengths:
    pages_append   gives each request the pages its new tokens need (a prompt at first,
                   then one token a step);
    slot_map       says where these tokens go in the cache;
    the model      writes their keys into the cache and makes logits (here: an embedding for a
                   key, and one matrix on the sum of the request's cached keys, read back
                   through the block table and divided by the root of their number);
    sample_tokens  picks a token a request;
    pages_release  puts the pages of finished requests back on the free list.
Everything stays on the GPU; the loop reads nothing back until its end.  A request that is
not granted its pages waits for the next step.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import prefix_scan_stream_amd as ps


def serve(requests=64, steps=40, page_size=16, vocab=4096, width=64, pages=None, longest=120, seed=0, on_step=None):
    """Runs the loop; returns (tokens of the last step, lengths, tables, free pages, free count, generated).
    on_step, where given, gets each step's (request of each new key, key, sums of the requests' cached keys,
    finished requests)."""
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    columns = -(-(longest + steps + 1) // page_size)
    pages = max(columns, requests * columns // 2) if pages is None else pages
    # whole numbers, so that their sums do not depend on the order of the additions
    embed = torch.randint(-2, 3, (vocab, width), device=dev, generator=g).float()
    head = torch.randn(width, vocab, device=dev, generator=g) * 0.4
    # a slot more than the pages have: the keys of entries that are no token go there
    keys = torch.zeros(pages * page_size + 1, width, device=dev)
    spare = pages * page_size
    at = torch.arange(columns * page_size, device=dev)
    tables = torch.full((requests, columns), -1, dtype=torch.int32, device=dev)
    free = torch.arange(pages, dtype=torch.int32, device=dev)
    count = torch.full((1,), pages, device=dev)
    lens = torch.zeros(requests, dtype=torch.int32, device=dev)
    prompt = torch.randint(1, longest + 1, (requests,), dtype=torch.int32, device=dev, generator=g)
    tokens = torch.randint(0, vocab, (requests,), device=dev, generator=g)
    generated = torch.zeros(requests, dtype=torch.int64, device=dev)
    temperature = torch.rand(requests, device=dev, generator=g) * 0.8 + 0.4
    top_k = torch.full((requests,), 50, dtype=torch.int32, device=dev)
    top_p = torch.full((requests,), 0.95, device=dev)
    room = requests * (longest + 1)

    for _ in range(steps):
        # the prompt of a request that holds nothing yet, else the token of the last step
        new = torch.where(lens == 0, prompt, torch.ones_like(lens))
        count, granted = ps.pages_append(lens, new, tables, free, count, page_size)
        new = torch.where(granted, new, torch.zeros_like(new))
        slots, positions, owner, offsets = ps.slot_map(lens, new, tables, page_size, room)
        live = slots >= 0
        rows = owner.clamp_min(0).long()
        x = embed[(tokens[rows] + positions) % vocab] * live[:, None]
        keys.index_copy_(0, torch.where(live, slots, torch.full_like(slots, spare)), x)
        lens = lens + new
        cached = tables[:, at // page_size].long() * page_size + at % page_size
        sums = keys[torch.where(at < lens[:, None], cached, torch.full_like(cached, spare))].sum(1)
        logits = (sums / lens.clamp_min(1)[:, None].float().sqrt()) @ head
        uniforms = torch.rand(requests, device=dev, generator=g)
        picked, _ = ps.sample_tokens(logits, uniforms, temperature, top_k=top_k, top_p=top_p)
        tokens = torch.where(granted, picked, tokens)
        generated += granted
        # a token in eight ends its request; its row starts over with another prompt
        done = granted & (tokens % 8 == 0)
        count = ps.pages_release(lens, done, tables, free, count, page_size)
        tables.masked_fill_(done[:, None], -1)
        lens = lens.masked_fill(done, 0)
        if on_step is not None:
            on_step(owner, x, sums, done)
    return tokens, lens, tables, free, count, generated


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--page-size", type=int, default=16)
    a = ap.parse_args()
    _, lens, tables, free, count, generated = serve(a.requests, a.steps, a.page_size)
    print(f"{int(generated.sum())} tokens in {a.steps} steps; {int((tables >= 0).sum())} pages in use, "
          f"{int(count)} free, longest request {int(lens.max())} tokens")


if __name__ == "__main__":
    main()
