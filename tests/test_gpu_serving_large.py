"""Serving calls of more work than the SMs take at once, against 64-bit implementations on the GPU."""
import numpy as np
import pytest
import torch

import serving_model as model
from paged_kv_cache_compose_gb300 import cpkv
from paged_kv_cache_compose_gb300.runtime import PagedCache
from test_gpu_serving import BF16, FP16, page_tables

pytestmark = pytest.mark.gpu


def randn(gen, *shape, dtype, factor=1.0):
    return (torch.randn(shape, device="cuda", generator=gen) * factor).to(dtype)


def pools_of(gen, n_pages, ps, cp, width, dtype):
    return [randn(gen, -(-(n_pages + 1) // cp), ps, width, dtype=dtype) for _ in range(cp)]


def rows_of(pools, pages, n):
    """Token rows 0 .. n - 1 of a page list, in 64 bits."""
    cp, ps = len(pools), pools[0].shape[1]
    t = torch.arange(n)
    pages = torch.as_tensor(np.asarray(pages)[: -(-n // ps)].astype(np.int64))
    flat = torch.stack(pools)  # [cp, cap, ps, width]
    page = pages[t // ps].cuda()
    return flat[page % cp, page // cp, (t % ps).cuda()].double()


def softmax(q, rows, sees, hkv, scale):
    """[tokens, heads, d] queries over [keys, 2 * hkv * d] rows, sees [tokens, keys] or None: output, log-sum-exp, weighted |values|."""
    n, heads, d = q.shape
    k, v = rows.unflatten(1, (2, hkv, d)).unbind(1)
    q = q.double().unflatten(1, (hkv, heads // hkv))
    s = torch.einsum("thgd,khd->thgk", q, k) * scale
    if sees is not None:
        s = s.masked_fill(~sees[:, None, None], -torch.inf)
    lse = torch.logsumexp(s, -1) if s.shape[-1] else torch.full(s.shape[:-1], -torch.inf, dtype=torch.float64, device="cuda")
    w = torch.exp(s - lse.nan_to_num(neginf=0.0)[..., None])
    return tuple(x.flatten(1, 2).cpu() for x in (torch.einsum("thgk,khd->thgd", w, v), lse, torch.einsum("thgk,khd->thgd", w, v.abs())))


def joined(parts):
    return tuple(torch.cat(x) for x in zip(*parts))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("axes, dtype", [(1, FP16), (3, BF16)])
def test_append_of_many_tokens(interleaved, axes, dtype):
    """Two heads (and value chunks) a thread, of odd numbers, and several units for every thread of the grid."""
    n, hq, hkv, dk, dv, rot, ps, cp, most = 40_000, 6, 1, 64, 72, 48, 16, 3, 5000
    gen = torch.Generator(device="cuda").manual_seed(axes)
    pages = -(-n // ps) + 40
    pools = pools_of(gen, pages, ps, cp, hkv * (dk + dv), dtype)
    assert n * ((hq + hkv) * 4 + hkv * dv // 8) > 2 * 2048 * torch.cuda.get_device_properties(0).multi_processor_count
    slots = ps + torch.randperm(pages * ps, device="cuda", generator=gen)[:n]
    slots[::9] = -1
    positions = torch.randint(0, most, (axes, n), device="cuda", generator=gen, dtype=torch.int32)
    axis = [(0, 1, 2, 1)[i % 4] if axes > 1 else 0 for i in range(rot // 2)]  # changing within four frequencies
    angle = torch.rand(most, rot // 2, device="cuda", generator=gen, dtype=torch.float64) * 6 - 3
    table = torch.cat([angle.cos(), angle.sin()], 1).float()
    k, v, q = (randn(gen, n, h, d, dtype=dtype, factor=1.5) for h, d in ((hkv, dk), (hkv, dv), (hq, dk)))
    cache = PagedCache([p.clone() for p in pools], page_size=ps, kv_heads=hkv, key_dim=dk, value_dim=dv)
    got = cache.append_rotary(k, v, slots, positions if axes > 1 else positions[0], table, q=q, interleaved=interleaved,
                              axis_of_freq=axis if axes > 1 else None)
    assert int(cache.d_status) == 0

    of = positions[torch.tensor(axis, device="cuda")].long().T  # [n, rot / 2]
    freq = torch.arange(rot // 2, device="cuda")
    turn = torch.complex(table[of, freq].double(), table[of, rot // 2 + freq].double())[:, None]

    def turned(x):
        y = x.double()
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(y[..., a].clone(), y[..., b].clone()) * turn
        y[..., a], y[..., b] = z.real, z.imag
        return y

    def close(got, want):  # one rounding of a sum of two 32-bit products of values below 10: half a step, and 2^-20 for the products
        return bool(((got.double() - want).abs() <= model.bound_of(dtype) * want.abs() + 2.0**-20).all())

    assert close(got, turned(q))
    want = torch.stack(pools).double()
    keep = slots >= 0
    page, row = slots[keep] // ps, slots[keep] % ps
    want[page % cp, page // cp, row] = torch.cat([turned(k).flatten(1), v.double().flatten(1)], 1)[keep]
    assert close(torch.stack(cache.table.pools), want)


WINDOWS = [  # heads, kv heads, dim, ps, dtype, window, sinks
    (32, 8, 64, 16, BF16, 0, 0),
    (32, 8, 128, 64, FP16, 200, 5),
    (40, 8, 64, 1, FP16, 90, 130),
    (24, 8, 128, 48, BF16, 0, 0),
]


def window_result(case, q_lens, kv_lens, seed):
    hq, hkv, d, ps, dtype, window, sinks = case
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lists, n_pages = page_tables(rng, kv_lens, ps)
    pools = pools_of(gen, n_pages, ps, 2, 2 * hkv * d, dtype)
    q = randn(gen, sum(q_lens), hq, d, dtype=dtype, factor=1.5)
    cache = PagedCache(pools, page_size=ps, kv_heads=hkv, key_dim=d)
    args = q, q_lens, torch.from_numpy(lists).cuda(), torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    results = []
    for _ in range(2):
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        results.append((cache.attend_window(*args, max_kv_len=max(kv_lens), window=window, sinks=sinks, lse=lse), lse))
    assert int(cache.d_status) == 0
    (out, lse), again = results
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    parts, t = [], 0
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        p = kv - n + torch.arange(n, device="cuda")[:, None]
        j = torch.arange(kv, device="cuda")
        sees = (j <= p) & ((p - j < window) | (j < sinks) if window else torch.ones((), dtype=torch.bool, device="cuda"))
        parts.append(softmax(q[t:t + n], rows_of(pools, lists[b], kv), sees, hkv, d**-0.5))
        t += n
    model.check(out, lse, joined(parts), dtype)
    return cache


@pytest.mark.parametrize("case", WINDOWS, ids=lambda c: "-".join(map(str, c)))
def test_window_of_many_more_items_than_sms(case):
    """Requests of a few query rows, of one item's rows and of many, empty ones among them: every block works through several items of
    one and of two streams."""
    q_lens = [300, 5, 0, 64, 17, 1, 130, 33, 2, 257] * 5
    kv_lens = [n + (37 * i) % 400 for i, n in enumerate(q_lens)]
    kv_lens[3], kv_lens[10] = 40, 0  # shorter than the queries
    tiles = sum(-(-n * case[0] // case[1] // 256) for n in q_lens)
    assert tiles * case[1] > 4 * torch.cuda.get_device_properties(0).multi_processor_count
    window_result(case, q_lens, kv_lens, case[2])


@pytest.mark.parametrize("case", WINDOWS, ids=lambda c: "-".join(map(str, c)))
def test_window_of_many_items_in_parts(case):
    """A few more items than SMs over long keys: each in parts, which make several rounds of blocks."""
    case = (*case[:5], 0, 0)
    q_lens = [9, 31, 12, 40, 6] * 4
    kv_lens = [n + 9000 + (1711 * i) % 9000 for i, n in enumerate(q_lens)]
    assert cpkv.cpkv_attend_window_workspace_bytes(20, case[0], case[1], case[2], q_lens, max(kv_lens)) > 0
    window_result(case, q_lens, kv_lens, case[2])


@pytest.mark.parametrize("case", WINDOWS, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("sizes, prefix", [([100, 0, 3, 57], [960, 48, 0, 2400]), ([2] * 70, [96] * 70)], ids=["groups", "pairs"])
def test_shared_of_many_more_items_than_sms(case, sizes, prefix):
    hq, hkv, d, ps, dtype, _, _ = case
    if hq // hkv * max(sizes) <= 16:
        hkv = 2  # more rows than the split kernel takes
    requests = sum(sizes)
    suffix = [(29 * i) % 300 for i in range(requests)]
    prefix = [n // ps * ps for n in prefix]
    rng = np.random.default_rng(requests)
    gen = torch.Generator(device="cuda").manual_seed(requests)
    lists, n_pages = page_tables(rng, prefix + suffix, ps)
    pools = pools_of(gen, n_pages, ps, 2, 2 * hkv * d, dtype)
    prefix_pages = np.concatenate([lists[g, :n // ps] for g, n in enumerate(prefix)]).astype(np.int32)
    q = randn(gen, requests, hq, d, dtype=dtype, factor=1.5)
    cache = PagedCache(pools, page_size=ps, kv_heads=hkv, key_dim=d)
    lse = torch.full((requests, hq), 7.0, device="cuda")
    out = cache.attend_shared(q, sizes, prefix, torch.from_numpy(prefix_pages).cuda(), torch.from_numpy(lists[len(sizes):]).cuda(),
                              torch.tensor(suffix, dtype=torch.int32, device="cuda"), max_suffix_len=max(suffix), lse=lse)
    assert int(cache.d_status) == 0
    parts, b = [], 0
    for g, n in enumerate(sizes):
        before = rows_of(pools, lists[g], prefix[g])
        for r in range(b, b + n):
            parts.append(softmax(q[r:r + 1], torch.cat([before, rows_of(pools, lists[len(sizes) + r], suffix[r])]), None, hkv, d**-0.5))
        b += n
    model.check(out, lse, joined(parts), dtype)
