"""One layer of a small serving loop: a prefill over a composed dense buffer, then decode steps over the pools.

Requests share a prompt's pages.  Their own first tokens are rotated into rows
(append_rotary), composed behind the prefix (compose_fused) and attended to in
the dense buffer (attend_window); the same rows go to the pools, where each
decode step appends a token per request and attends to the shared prompt once
(attend_shared) and to each request's own rows.  With quantised rows (QuantisedCache) the same calls
work on half the bytes.

    python examples/serving_step.py [--quantised]
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from paged_kv_cache_compose_gb300.runtime import ComposeLayers, ComposePlan, PagedCache, QuantisedCache  # noqa: E402

PAGE, OWNERS, HEADS, KV_HEADS, DIM = 16, 2, 8, 2, 64
PREFIX, OWN, STEPS = 64, [20, 5, 33], 3  # prompt tokens, each request's own tokens, decode steps


def rope_table(positions: int, dim: int, device) -> torch.Tensor:
    """Cosines, then sines, of position * 10000^(-2 i / dim)."""
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


def random_heads(gen, tokens: int, heads: int, device) -> torch.Tensor:
    return torch.randn(tokens, heads, DIM, generator=gen).to(torch.bfloat16).to(device)


def run(seed: int = 0, device: str = "cuda", quantised: bool = False) -> dict:
    """The loop's inputs and results, for a check from outside."""
    gen = torch.Generator().manual_seed(seed)
    requests = len(OWN)
    if quantised:
        Cache, dtype, width = QuantisedCache, torch.uint8, QuantisedCache.row_bytes(KV_HEADS, DIM)
    else:
        Cache, dtype, width = PagedCache, torch.bfloat16, 2 * KV_HEADS * DIM
    turns = rope_table(PREFIX + max(OWN) + STEPS, DIM, device)
    # pages: the prompt's, then each request's own with room for the decode steps
    prompt_pages = PREFIX // PAGE
    own_pages = [-(-(n + STEPS) // PAGE) for n in OWN]
    order = 1 + torch.randperm(prompt_pages + sum(own_pages), generator=gen)
    prompt, rest = order[:prompt_pages], order[prompt_pages:].split(own_pages)
    cap = int(order.max()) // OWNERS + 1
    pools = [torch.zeros(cap, PAGE, width, dtype=dtype, device=device) for _ in range(OWNERS)]
    cache = Cache(pools, page_size=PAGE, kv_heads=KV_HEADS, key_dim=DIM)
    table = torch.zeros(requests, max(own_pages), dtype=torch.int32)
    for b, pages in enumerate(rest):
        table[b, :len(pages)] = pages
    d_prompt, d_table = prompt.int().to(device), table.to(device)

    def slots(pages, first, n):
        t = torch.arange(first, first + n)
        return pages[t // PAGE] * PAGE + t % PAGE

    # the prompt's rows, once for all requests
    at = torch.arange(PREFIX, dtype=torch.int32, device=device)
    k, v = random_heads(gen, PREFIX, KV_HEADS, device), random_heads(gen, PREFIX, KV_HEADS, device)
    cache.append_rotary(k, v, slots(prompt, 0, PREFIX).to(device), at, turns)

    # prefill: each request's own tokens, as rows that the compose puts behind the prompt's pages
    total = sum(OWN)
    q, k, v = (random_heads(gen, total, h, device) for h in (HEADS, KV_HEADS, KV_HEADS))
    positions = torch.cat([PREFIX + torch.arange(n, dtype=torch.int32) for n in OWN]).to(device)
    rows = torch.empty(total, 1, width, dtype=dtype, device=device)
    writer = Cache([rows], page_size=1, kv_heads=KV_HEADS, key_dim=DIM, dense=True)
    q = writer.append_rotary(k, v, torch.arange(total, device=device), positions, turns, q=q)
    cur_pages = torch.cat([table[b, :-(-n // PAGE)] for b, n in enumerate(OWN)])
    plan = ComposePlan([PREFIX] * requests, OWN, prompt.repeat(requests).numpy(), cur_pages.numpy(), np.zeros(len(cur_pages), np.int32),
                       page_size=PAGE, cp_size=OWNERS, num_pool_pages=cap * OWNERS, device=device).build()
    layers = ComposeLayers(plan, rows[0].nbytes, num_dense=1)
    dense = layers.dense[0]
    layers.compose_fused([p.view(torch.uint8) for p in pools], [rows.view(torch.uint8).view(total, -1), dense[:0]], dense)
    composed = Cache([dense.view(dtype).view(-1, PAGE, width)], page_size=PAGE, kv_heads=KV_HEADS, key_dim=DIM, dense=True)
    pages = [prompt_pages + -(-n // PAGE) for n in OWN]
    dense_table = torch.zeros(requests, max(pages), dtype=torch.int32)
    for b, n in enumerate(pages):
        dense_table[b, :n] = sum(pages[:b]) + torch.arange(n)
    lens = torch.tensor([PREFIX + n for n in OWN], dtype=torch.int32, device=device)
    prefill = composed.attend_window(q, OWN, dense_table.to(device), lens, max_kv_len=PREFIX + max(OWN))

    # the same rows into the pools: attention there gives the same bits
    own_slots = torch.cat([slots(pages_, 0, n) for pages_, n in zip(rest, OWN)]).to(device)
    cache.append_rotary(k, v, own_slots, positions, turns)
    both = torch.cat([prompt.int().expand(requests, -1), table], 1).to(device)
    paged = cache.attend_window(q, OWN, both, lens, max_kv_len=PREFIX + max(OWN))

    # decode: a token per request and step
    suffix = torch.tensor(OWN, dtype=torch.int32, device=device)
    decode, window = [], []
    for step in range(STEPS):
        q1, k1, v1 = (random_heads(gen, requests, h, device) for h in (HEADS, KV_HEADS, KV_HEADS))
        new = torch.cat([slots(pages_, n + step, 1) for pages_, n in zip(rest, OWN)]).to(device)
        q1 = cache.append_rotary(k1, v1, new, PREFIX + suffix, turns, q=q1)
        suffix = suffix + 1
        decode.append(cache.attend_shared(q1, [requests], [PREFIX], d_prompt, d_table, suffix, max_suffix_len=max(OWN) + STEPS))
        window.append(cache.attend_window(q1, None, both, PREFIX + suffix, max_kv_len=PREFIX + max(OWN) + STEPS))
    torch.cuda.synchronize()
    status = [int(c.d_status) for c in (cache, writer, composed)] + [int(plan.d_status)]
    return dict(status=status, prefill=prefill, paged=paged, decode=decode, window=window)


if __name__ == "__main__":
    got = run(quantised="--quantised" in sys.argv[1:])
    assert not any(got["status"]), got["status"]
    assert torch.equal(got["prefill"], got["paged"])
    off = max(float((a.float() - b.float()).abs().max()) for a, b in zip(got["decode"], got["window"]))
    print(f"prefill over the dense buffer equals prefill over the pools; decode with and without sharing differ by {off:.2g}")
