"""The serving operators on the GPU against plain 64-bit implementations."""
import importlib.util
import math
import pathlib

import numpy as np
import pytest
import torch

import serving_model as model
from paged_kv_cache_compose_gb300 import cpkv
from paged_kv_cache_compose_gb300.runtime import PagedCache

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


def page_tables(rng, lens, ps, spare=0):
    """Random page lists of the requests, one row each (unused entries name no page), and the pages in use."""
    need = [-(-n // ps) for n in lens]
    perm = 1 + rng.permutation(sum(need) + spare)
    table = np.full((len(lens), max([1] + need)), 1 << 30, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, sum(need) + spare


def queries(rng, n, heads, dim, dtype, factor=1.5):
    return torch.from_numpy((factor * rng.standard_normal((n, heads, dim))).astype(np.float32)).to(dtype)


# --------------------------------------------------------------------------- append

APPEND = [  # n, q heads, kv heads, key dim, value dim, rot, interleaved, axes, ps, cp, dtype, (key offset, value offset, row elements)
    (1, 8, 1, 64, 64, 64, False, 1, 16, 1, BF16, None),
    (37, 4, 2, 128, 128, 128, False, 1, 16, 2, BF16, None),
    (37, 4, 2, 128, 128, 96, True, 1, 1, 8, FP16, None),
    (130, 5, 1, 64, 64, 32, False, 3, 64, 3, FP16, None),
    (65, 8, 8, 64, 64, 48, True, 3, 16, 2, BF16, None),
    (33, 16, 1, 64, 512, 64, True, 1, 16, 2, BF16, (512, 0, 576)),
    (33, 0, 2, 72, 40, 16, False, 1, 5, 2, BF16, (88, 0, 232)),
    (9, 3, 1, 256, 256, 256, False, 4, 7, 1, FP16, (264, 8, 528)),
    (20, 2, 1, 64, 64, 0, False, 1, 16, 2, BF16, None),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(map(str, c[:11])))
def test_append_matches_64_bits(case):
    n, hq, hkv, dk, dv, rot, interleaved, axes, ps, cp, dtype, layout = case
    k_at, v_at, width = layout or (0, hkv * dk, hkv * (dk + dv))
    rng = np.random.default_rng(n + rot)
    n_pages = -(-n // ps) + 3
    pools = model.Pools(rng, n_pages, ps, cp, width, dtype)
    slots = ps + rng.permutation(n_pages * ps)[:n]
    slots[::7] = np.where(np.arange(n)[::7] % 2 == 0, slots[::7], -1)  # some padding tokens
    max_pos = 500
    positions = rng.integers(0, max_pos, (axes, n)).astype(np.int32)
    axis = rng.integers(0, axes, rot // 2).tolist()
    angle = rng.uniform(-3, 3, (max_pos, rot // 2))
    table = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32))
    k, v = queries(rng, n, hkv, dk, dtype), queries(rng, n, hkv, dv, dtype)
    q = queries(rng, n, hq, dk, dtype) if hq else None
    want_q, want = model.append(pools, k, v, q, slots, positions, table, axis, interleaved, k_at, v_at)
    cache = PagedCache(pools.cuda(), page_size=ps, kv_heads=hkv, key_dim=dk, value_dim=dv, key_offset=k_at, value_offset=v_at)
    pos = torch.from_numpy(positions).cuda()
    got_q = cache.append_rotary(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), pos if axes > 1 else pos[0], table.cuda(),
                                q=None if q is None else q.cuda(), axis_of_freq=axis if axes > 1 else None, interleaved=interleaved)
    torch.cuda.synchronize()
    assert int(cache.d_status) == 0
    # one rounding of a sum of two 32-bit products of values below 8: half a step, and 2^-20 for the products
    u = model.bound_of(dtype)
    for got, ref in [(got_q, want_q)] * bool(hq) + list(zip(cache.table.pools, want)):
        got = got.double().cpu()
        assert bool(((got - ref).abs() <= u * ref.abs() + 2.0**-20).all())


def test_append_takes_slices_and_rotates_in_place():
    """Queries, keys and values as slices of one projection's output; the queries rotated where they stand."""
    rng = np.random.default_rng(5)
    n, hq, hkv, d, ps = 50, 4, 2, 64, 16
    qkv = queries(rng, n, hq + 2 * hkv, d, BF16).cuda()
    pools = model.Pools(rng, 8, ps, 2, 2 * hkv * d, BF16)
    slots = torch.from_numpy(ps + rng.permutation(8 * ps)[:n]).cuda()
    angle = rng.uniform(-3, 3, (100, d // 2))
    table = torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)).cuda()
    pos = torch.from_numpy(rng.integers(0, 100, n).astype(np.int32)).cuda()
    one = PagedCache(pools.cuda(), page_size=ps, kv_heads=hkv, key_dim=d)
    two = PagedCache(pools.cuda(), page_size=ps, kv_heads=hkv, key_dim=d)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    want = one.append_rotary(k.contiguous(), v.contiguous(), slots, pos, table, q=q.contiguous())
    two.append_rotary(k, v, slots, pos, table, q=q, q_out=q)
    assert torch.equal(q, want)
    for a, b in zip(one.table.pools, two.table.pools):
        assert torch.equal(a, b)


def test_append_reports_bad_slots_and_positions():
    """Rows whose page or position is out of range are not written; the others are."""
    rng = np.random.default_rng(6)
    ps, d = 4, 64
    pools = model.Pools(rng, 5, ps, 2, 2 * d, BF16)
    table = torch.ones(10, d, device="cuda")
    k, v, q = (queries(rng, 4, 1, d, BF16).cuda() for _ in range(3))
    for slots, pos, bit in [([4, 2, 8, 12], [0, 1, 2, 3], cpkv.STATUS_PAGE_OOB), ([4, 24, 8, 12], [0, 1, 2, 3], cpkv.STATUS_PAGE_OOB),
                            ([4, 1 << 40, 8, 12], [0, 1, 2, 3], cpkv.STATUS_PAGE_OOB),
                            ([4, 20, 8, 12], [0, 10, 2, 3], cpkv.STATUS_POS_OOB), ([4, 20, 8, 12], [0, -1, 2, 3], cpkv.STATUS_POS_OOB)]:
        cache = PagedCache(pools.cuda(), page_size=ps, kv_heads=1, key_dim=d)
        got = cache.append_rotary(k, v, torch.tensor(slots).cuda(), torch.tensor(pos, dtype=torch.int32).cuda(), table, q=q)
        assert int(cache.d_status) == bit
        assert bool((got[1] == 0).all()) == (bit == cpkv.STATUS_POS_OOB)
        for page in range(1, 6):
            new, old = cache.table.pools[page % 2][page // 2], pools.slabs[page % 2][page // 2].cuda()
            assert torch.equal(new[1:], old[1:])
            assert torch.equal(new[0], old[0]) == (page not in (1, 2, 3))


# --------------------------------------------------------------------------- window

WINDOW = [  # q heads, kv heads, dim, ps, cp, dtype, window, sinks, q lens, kv lens
    (4, 1, 64, 16, 1, BF16, 0, 0, [1], [1]),
    (4, 1, 128, 16, 2, FP16, 0, 0, [1], [777]),
    (8, 2, 128, 64, 8, BF16, 0, 0, [1, 1, 1, 1, 1], [1, 64, 65, 1000, 0]),
    (8, 2, 64, 16, 2, FP16, 100, 4, [1] * 6, [1, 3, 99, 104, 105, 900]),
    (5, 1, 64, 1, 3, BF16, 1, 0, [1] * 3, [1, 2, 130]),
    (7, 1, 128, 5, 2, BF16, 33, 200, [1] * 4, [10, 199, 234, 500]),
    (16, 1, 128, 16, 2, BF16, 0, 0, [1, 1], [300, 5]),
    (17, 1, 64, 16, 2, BF16, 40, 1, [1, 1], [300, 5]),
    (8, 2, 128, 16, 2, BF16, 0, 0, [3, 3, 3], [3, 50, 200]),
    (8, 2, 64, 16, 2, FP16, 20, 2, [4, 4, 4], [2, 50, 131]),  # a request shorter than its queries
    (4, 2, 64, 16, 2, BF16, 0, 0, [7, 0, 64, 1], [7, 20, 100, 33]),
    (4, 1, 128, 16, 2, BF16, 50, 3, [70, 33], [70, 133]),
    (2, 2, 128, 64, 4, FP16, 0, 0, [130], [300]),
    (8, 1, 64, 16, 2, BF16, 64, 64, [65, 1, 20], [65, 64, 129]),
    (4, 4, 64, 1, 1, BF16, 10, 0, [1, 2] * 10, [1, 2, 3, 4, 30] * 4),
    (4, 1, 128, 16, 2, BF16, 0, 0, [300], [340]),
    (6, 2, 64, 16, 2, FP16, 129, 5, [200, 90], [530, 90]),
    (40, 8, 128, 16, 2, BF16, 0, 0, [9], [20]),
]


def window_case(case, seed=0, poison=False):
    hq, hkv, d, ps, cp, dtype, w, sinks, q_lens, kv_lens = case
    rng = np.random.default_rng(seed + sum(kv_lens))
    table, n_pages = page_tables(rng, kv_lens, ps)
    pools = model.Pools(rng, n_pages, ps, cp, 2 * hkv * d, dtype)
    q = queries(rng, sum(q_lens), hq, d, dtype)
    return rng, pools, table, q


def run_window(cache, case, q, table, max_kv=None, **more):
    w, sinks, q_lens, kv_lens = case[6:]
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out = cache.attend_window(q.cuda(), None if all(n == 1 for n in q_lens) else q_lens, torch.from_numpy(table).cuda(),
                              torch.tensor(kv_lens, dtype=torch.int32).cuda(),
                              max_kv_len=max(kv_lens) if max_kv is None else max_kv, window=w, sinks=sinks, lse=lse, **more)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("case", WINDOW, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c)[:80])
def test_window_matches_64_bits(case):
    hq, hkv, d, ps, cp, dtype, w, sinks, q_lens, kv_lens = case
    rng, pools, table, q = window_case(case)
    want = model.window(q, q_lens, table, kv_lens, pools, kv_heads=hkv, dim=d, window=w, sinks=sinks, scale=d**-0.5)
    cache = PagedCache(pools.cuda(), page_size=ps, kv_heads=hkv, key_dim=d)
    out, lse = run_window(cache, case, q, table)
    assert int(cache.d_status) == 0
    model.check(out, lse, want, dtype)
    again, lse2 = run_window(cache, case, q, table)
    assert torch.equal(out, again) and torch.equal(lse, lse2)  # the same bits every time


@pytest.mark.parametrize("case", [c for c in WINDOW if c[6]], ids=lambda c: "-".join(str(x).replace(" ", "") for x in c)[:80])
def test_window_reads_nothing_that_no_query_sees(case):
    """Rows behind the window and past the length hold NaN, and pages wholly there have no page id."""
    hq, hkv, d, ps, cp, dtype, w, sinks, q_lens, kv_lens = case
    rng, pools, table, q = window_case(case)
    cache = PagedCache(pools.cuda(), page_size=ps, kv_heads=hkv, key_dim=d)
    want, want_lse = run_window(cache, case, q, table)
    for b, (nq, kv) in enumerate(zip(q_lens, kv_lens)):
        first = max(0, kv - nq - w + 1)
        for page in range(-(-kv // ps)):
            seen = [nq > 0 and t < kv and (t >= first or t < min(sinks, first)) for t in range(page * ps, page * ps + ps)]
            lp = int(table[b, page])
            pools.slabs[lp % cp][lp // cp][~torch.tensor(seen)] = float("nan")
            if not any(seen):
                table[b, page] = -5
    poisoned = PagedCache(pools.cuda(), page_size=ps, kv_heads=hkv, key_dim=d)
    out, lse = run_window(poisoned, case, q, table)
    assert int(poisoned.d_status) == 0
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


MIXED = [c for c in WINDOW if max(c[8]) > 1] + [
    (1, 1, 128, 16, 2, BF16, 0, 0, [256, 100], [700, 100]),  # 256 tokens an item: several tiles that only some see
    (1, 1, 64, 7, 2, FP16, 140, 130, [300], [900]),
    (64, 1, 128, 32, 2, FP16, 6, 0, [9], [300]),  # every row sees a NaN among its keys
    (64, 1, 128, 32, 2, FP16, 60, 0, [9], [300]),
    (16, 2, 64, 16, 2, BF16, 0, 0, [5], [2600]),  # two streams, parts
]


@pytest.mark.parametrize("case", MIXED, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c)[:80])
def test_window_infinite_values_reach_only_the_rows_that_see_them(case):
    """Keys and values that hold infinities and NaNs where some query tokens of the request see them and others do not."""
    hq, hkv, d, ps, cp, dtype, w, sinks, q_lens, kv_lens = case
    rng, pools, table, q = window_case(case)
    for b, (nq, kv) in enumerate(zip(q_lens, kv_lens)):
        edge = kv - nq - (w or 10**6) + nq // 2
        for j, what, key in [(kv - 1, math.inf, False), (kv - nq // 3 - 1, math.nan, False), (kv - nq // 2, math.nan, True),
                             (edge, -math.inf, False), (edge + 1, math.nan, True)]:
            if 0 <= j < kv:
                pools.row(int(table[b, j // ps]), j % ps)[rng.integers(0, d) + (0 if key else hkv * d)] = what
    want = model.window(q, q_lens, table, kv_lens, pools, kv_heads=hkv, dim=d, window=w, sinks=sinks, scale=d**-0.5)
    cache = PagedCache(pools.cuda(), page_size=ps, kv_heads=hkv, key_dim=d)
    out, lse = run_window(cache, case, q, table)
    assert int(cache.d_status) == 0
    finite = want[0].isfinite()
    assert not finite.all()
    assert torch.equal(out.cpu().isfinite(), finite)
    seen = [torch.where(finite, x, 0.0) for x in (out.double().cpu(), want[0], want[2])]
    model.check(seen[0], None, (seen[1], want[1], seen[2]), dtype)
    assert torch.equal(lse.cpu().isnan(), want[1].isnan())


@pytest.mark.parametrize("rows", [1, 40])
def test_window_scores_that_grow_and_infinite_scores(rows):
    """Keys whose scores rise along the sequence by far more than a 32-bit exponential holds, then one score of -infinity."""
    rng = np.random.default_rng(8)
    d, ps, kv = 128, 16, 900
    case = (4, 1, d, ps, 2, BF16, 0, 0, [rows], [kv])
    _, pools, table, q = window_case(case)
    q.zero_()
    q[..., 0] = 16.0
    for t in range(kv):
        pools.row(int(table[0, t // ps]), t % ps)[0] = t // 7  # scores up to 16 * 128 / sqrt(128)
    pools.row(int(table[0, 0]), 3)[0] = -float("inf")
    want = model.window(q, [rows], table, [kv], pools, kv_heads=1, dim=d, window=0, sinks=0, scale=d**-0.5)
    cache = PagedCache(pools.cuda(), page_size=ps, kv_heads=1, key_dim=d)
    out, lse = run_window(cache, case, q, table)
    got = out.double().cpu()
    # scores of about 200 carry 32-bit errors of 2^-16 each: the bound on the weights grows by as much
    u = model.bound_of(BF16)
    assert bool(((got - want[0]).abs() <= u * want[0].abs() + (u + 2.0**-10) * want[2] + 2.0**-24).all())
    assert float((lse.double().cpu() - want[1]).abs().max()) <= 2.0**-10


@pytest.mark.parametrize("nq", [1, 3, 50])
def test_window_reports_bad_pages_and_lengths(nq):
    """A bad page id reads as zero rows, a length past the bound is clamped; both raise their bit."""
    case = (4, 1, 64, 16, 2, BF16, 0, 0, [nq, nq], [100, 60])
    rng, pools, table, q = window_case(case)
    good = table.copy()
    for bad in (-1, 0, 1 << 29):
        table[0, 2] = bad
        cache = PagedCache(pools.cuda(), page_size=16, kv_heads=1, key_dim=64)
        out, lse = run_window(cache, case, q, table)
        assert int(cache.d_status) == cpkv.STATUS_PAGE_OOB
        zeroed = model.Pools(np.random.default_rng(0), 1, 16, 2, 128, BF16)
        zeroed.slabs = [s.clone() for s in pools.slabs]
        lp = int(good[0, 2])
        zeroed.slabs[lp % 2][lp // 2] = 0
        want = model.window(q, [nq, nq], good, [100, 60], zeroed, kv_heads=1, dim=64, window=0, sinks=0, scale=0.125)
        model.check(out, lse, want, BF16)
    cache = PagedCache(pools.cuda(), page_size=16, kv_heads=1, key_dim=64)
    out, lse = run_window(cache, case, q, good, max_kv=90)
    assert int(cache.d_status) == cpkv.STATUS_OUT_CAPACITY
    model.check(out, lse, model.window(q, [nq, nq], good, [90, 60], pools, kv_heads=1, dim=64, window=0, sinks=0, scale=0.125), BF16)
    cache = PagedCache(pools.cuda(), page_size=16, kv_heads=1, key_dim=64)
    lens = torch.tensor([-3, 60], dtype=torch.int32).cuda()
    out = cache.attend_window(q.cuda(), [nq, nq], torch.from_numpy(good).cuda(), lens, max_kv_len=100)
    assert int(cache.d_status) == cpkv.STATUS_OUT_CAPACITY and bool((out[:nq] == 0).all())


@pytest.mark.parametrize("nq", [1, 33])
def test_window_strides_layouts_and_dense_pages(nq):
    """Queries and outputs as slices, rows with the values first and room between, one dense buffer whose page 0 counts."""
    rng = np.random.default_rng(9)
    hq, hkv, d, ps, kv = 6, 2, 64, 16, 150
    width = 2 * hkv * d + 24
    dense = torch.from_numpy(rng.standard_normal((10, ps, width)).astype(np.float32)).to(BF16)
    pools = model.Pools(rng, 9, ps, 1, width, BF16)
    pools.slabs = [dense]
    table = np.arange(10, dtype=np.int32)[None]
    wide = queries(rng, nq, hq + 4, d, BF16).cuda()
    q = wide[:, 2:2 + hq]
    holder = torch.zeros(nq, hq + 1, d, dtype=BF16, device="cuda")
    cache = PagedCache([dense.cuda()], page_size=ps, kv_heads=hkv, key_dim=d, key_offset=hkv * d + 16, value_offset=8, dense=True)
    lse = torch.empty(nq, hq, device="cuda")
    out = cache.attend_window(q, [nq], torch.from_numpy(table).cuda(), torch.tensor([kv], dtype=torch.int32).cuda(),
                              max_kv_len=kv, window=70, sinks=3, scale=0.3, out=holder[:, :hq], lse=lse)
    assert int(cache.d_status) == 0 and bool((holder[:, hq] == 0).all())
    want = model.window(q.cpu(), [nq], table, [kv], pools, kv_heads=hkv, dim=d, window=70, sinks=3, scale=0.3, k_at=hkv * d + 16, v_at=8)
    model.check(out, lse, want, BF16)


def test_window_in_a_graph_follows_the_lengths():
    """A captured decode step replayed on another stream as the requests grow."""
    case = (8, 2, 128, 16, 2, BF16, 100, 4, [1] * 3, [300, 90, 200])
    rng, pools, table, q = window_case(case)
    cache = PagedCache(pools.cuda(), page_size=16, kv_heads=2, key_dim=128)
    lens = torch.tensor([1, 1, 1], dtype=torch.int32).cuda()
    d_q, d_table = q.cuda(), torch.from_numpy(table).cuda()
    out, lse = torch.empty_like(d_q), torch.empty(3, 8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cache.attend_window(d_q, None, d_table, lens, max_kv_len=300, window=100, sinks=4, out=out, lse=lse)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        cache.attend_window(d_q, None, d_table, lens, max_kv_len=300, window=100, sinks=4, out=out, lse=lse)
    for now in ([300, 90, 200], [5, 0, 104]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = model.window(q, [1] * 3, table, now, pools, kv_heads=2, dim=128, window=100, sinks=4, scale=128**-0.5)
        model.check(out, lse, want, BF16, str(now))
    assert int(cache.d_status) == 0


def test_long_cache_offsets_past_32_bits():
    """Pages beyond 4 GB of one pool."""
    ps, hkv, d = 64, 8, 128
    pages = (5 << 30) // (ps * 2 * hkv * d * 2)
    pool = torch.zeros(pages, ps, 2 * hkv * d, dtype=BF16, device="cuda")
    rng = np.random.default_rng(4)
    pool[-2:] = torch.from_numpy(rng.standard_normal((2, ps, 2 * hkv * d)).astype(np.float32)).to(BF16).cuda()
    small = model.Pools(rng, 2, ps, 1, 2 * hkv * d, BF16)
    small.slabs = [torch.cat([pool[:1], pool[-2:]]).cpu()]
    for nq in (1, 40):
        q = queries(rng, nq, hkv, d, BF16)
        cache = PagedCache([pool], page_size=ps, kv_heads=hkv, key_dim=d)
        table = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32).cuda()
        lse = torch.empty(nq, hkv, device="cuda")
        out = cache.attend_window(q.cuda(), [nq], table, torch.tensor([100], dtype=torch.int32).cuda(), max_kv_len=128, lse=lse)
        want = model.window(q, [nq], [[1, 2]], [100], small, kv_heads=hkv, dim=d, window=0, sinks=0, scale=d**-0.5)
        model.check(out, lse, want, BF16)
    k = queries(rng, 1, hkv, d, BF16).cuda()
    cache.append_rotary(k, k, torch.tensor([(pages - 1) * ps + 5]).cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"),
                        torch.cat([torch.ones(1, 64), torch.zeros(1, 64)], 1).cuda())
    assert torch.equal(pool[-1, 5], torch.cat([k.flatten(), k.flatten()]))


# --------------------------------------------------------------------------- shared

SHARED = [  # q heads, kv heads, dim, ps, cp, dtype, group sizes, prefix lens, suffix lens
    (4, 1, 64, 16, 2, BF16, [1], [16], [1]),
    (8, 2, 128, 16, 2, BF16, [4], [512], [1, 30, 64, 17]),
    (8, 1, 64, 1, 3, FP16, [3, 0, 2], [77, 5, 201], [1, 2, 3, 100, 65]),
    (5, 1, 128, 64, 8, BF16, [2, 3], [0, 640], [10, 0, 1, 129, 64]),  # no prefix; no suffix
    (4, 2, 64, 16, 2, BF16, [2], [0], [0, 5]),  # nothing at all
    (16, 1, 128, 16, 2, FP16, [20], [304], [1 + 3 * i for i in range(20)]),
    (8, 8, 64, 16, 2, BF16, [1] * 18, [16 * i for i in range(18)], [2 + i for i in range(18)]),
    (14, 2, 64, 16, 2, BF16, [40], [160], [1 + i % 5 for i in range(40)]),
    (8, 2, 128, 16, 1, BF16, [70], [1040], [1 + i % 3 for i in range(70)]),
]


@pytest.mark.parametrize("case", SHARED, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c)[:80])
def test_shared_matches_64_bits(case):
    hq, hkv, d, ps, cp, dtype, sizes, prefix, suffix = case
    rng = np.random.default_rng(sum(suffix))
    lists, n_pages = page_tables(rng, prefix + suffix, ps)
    pools = model.Pools(rng, n_pages, ps, cp, 2 * hkv * d, dtype)
    prefix_pages = np.concatenate([lists[g, :n // ps] for g, n in enumerate(prefix)]).astype(np.int32)
    table = lists[len(prefix):]
    q = queries(rng, sum(sizes), hq, d, dtype)
    want = model.shared(q, sizes, prefix, prefix_pages, table, suffix, pools, kv_heads=hkv, dim=d, scale=d**-0.5)
    cache = PagedCache(pools.cuda(), page_size=ps, kv_heads=hkv, key_dim=d)
    results = []
    for _ in range(2):
        lse = torch.full((len(suffix), hq), 7.0, device="cuda")
        out = cache.attend_shared(q.cuda(), sizes, prefix, torch.from_numpy(prefix_pages).cuda(), torch.from_numpy(table).cuda(),
                                  torch.tensor(suffix, dtype=torch.int32).cuda(), max_suffix_len=max(suffix), lse=lse)
        torch.cuda.synchronize()
        results.append((out, lse))
    assert int(cache.d_status) == 0
    model.check(*results[0], want, dtype)
    assert torch.equal(results[0][0], results[1][0]) and torch.equal(results[0][1], results[1][1])


def test_shared_reports_bad_pages():
    rng = np.random.default_rng(3)
    pools = model.Pools(rng, 20, 16, 2, 128, BF16)
    cache = PagedCache(pools.cuda(), page_size=16, kv_heads=1, key_dim=64)
    q = queries(rng, 2, 2, 64, BF16).cuda()
    lens = torch.tensor([3, 4], dtype=torch.int32).cuda()
    table = torch.tensor([[5], [6]], dtype=torch.int32).cuda()
    for prefix_pages in ([1, 1000], [0, 2], [-1, 2]):
        cache.d_status.zero_()
        cache.attend_shared(q, [2], [32], torch.tensor(prefix_pages, dtype=torch.int32).cuda(), table, lens, max_suffix_len=16)
        assert int(cache.d_status) == cpkv.STATUS_PAGE_OOB


@pytest.mark.parametrize("case", [
    (48, 1, 64, 16, 2, FP16, [3, 1], [208, 64], [40, 3, 1, 90]),  # 48 heads to one: suffixes of several row tiles, few rows
    (160, 1, 64, 16, 2, BF16, [2], [400], [5, 200]),  # two row tiles of a single request's 160 heads
    (300, 1, 128, 32, 2, BF16, [1, 1], [96, 1024], [70, 1]),  # more heads than an item has rows
    (8, 1, 128, 1, 3, FP16, [24], [700], [1 + 11 * i for i in range(24)]),  # pages of one token, key by key
], ids=lambda c: "-".join(str(x).replace(" ", "") for x in c)[:80])
def test_shared_with_many_heads_to_one(case):
    test_shared_matches_64_bits(case)


@pytest.mark.parametrize("case", [
    (20, 1, 64, 16, 2, FP16, 0, 0, [1, 1], [700, 64]),  # several row tiles of one token
    (160, 1, 64, 48, 2, BF16, 0, 0, [1], [1500]),  # pages of 48 tokens: boxes of 16 rows
    (300, 1, 128, 32, 2, BF16, 90, 7, [1, 2], [1030, 400]),  # more heads than an item has rows
    (12, 1, 128, 128, 2, BF16, 0, 0, [11], [4000]),  # few rows over long keys: parts of two streams
    (4, 1, 64, 16, 12, FP16, 0, 0, [40], [600]),  # more pools than maps
], ids=lambda c: "-".join(str(x).replace(" ", "") for x in c)[:80])
def test_window_with_many_heads_to_one(case):
    test_window_matches_64_bits(case)


def test_shared_in_a_graph_follows_the_suffixes():
    """A captured decode step of two groups, replayed as the suffixes grow; a call of another size between."""
    rng = np.random.default_rng(11)
    ps, d, hkv, hq = 16, 64, 2, 8
    sizes, prefix, most = [12, 3], [160, 32], 80
    lists, n_pages = page_tables(rng, prefix + [most] * 15, ps)
    pools = model.Pools(rng, n_pages, ps, 2, 2 * hkv * d, BF16)
    prefix_pages = np.concatenate([lists[g, :n // ps] for g, n in enumerate(prefix)]).astype(np.int32)
    q = queries(rng, 15, hq, d, BF16)
    cache = PagedCache(pools.cuda(), page_size=ps, kv_heads=hkv, key_dim=d)
    d_q, d_table, d_prefix = q.cuda(), torch.from_numpy(lists[2:]).cuda(), torch.from_numpy(prefix_pages).cuda()
    lens = torch.ones(15, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(d_q), torch.empty(15, hq, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        cache.attend_shared(d_q, sizes, prefix, d_prefix, d_table, lens, max_suffix_len=most, out=out, lse=lse)

    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    with torch.cuda.stream(side):  # a larger call on the stream: the captured one keeps its own workspace
        cache.attend_window(queries(rng, 64, hq, d, BF16).cuda(), [64], d_table[:1], lens[:1] * 64, max_kv_len=most)
    side.synchronize()
    for now in ([1 + 5 * i for i in range(15)], [80 - i for i in range(15)]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        model.check(out, lse, model.shared(q, sizes, prefix, prefix_pages, lists[2:], now, pools, kv_heads=hkv, dim=d, scale=0.125), BF16)
    assert int(cache.d_status) == 0


def test_calls_refuse_what_their_tensors_cannot_be():
    """Types, widths, strides and counts of tensors that a call would read past or misread."""
    d, ps = 64, 16
    cache = PagedCache([torch.zeros(4, ps, 4 * d, dtype=BF16, device="cuda")], page_size=ps, kv_heads=2, key_dim=d)
    q = torch.zeros(3, 4, d, dtype=BF16, device="cuda")
    k = torch.zeros(3, 2, d, dtype=BF16, device="cuda")
    slots, pos = torch.arange(16, 19, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    turns = torch.ones(8, d, device="cuda")
    table, lens = torch.ones(3, 2, dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")

    def append(**changed):
        a = {**dict(k=k, v=k, slots=slots, positions=pos, cos_sin=turns), **changed}
        return cache.append_rotary(a.pop("k"), a.pop("v"), a.pop("slots"), a.pop("positions"), a.pop("cos_sin"), **a)

    def window(**changed):
        a = {**dict(q=q, q_lens=None, table=table, lens=lens, max_kv_len=32), **changed}
        return cache.attend_window(a.pop("q"), a.pop("q_lens"), a.pop("table"), a.pop("lens"), **a)

    def shared(**changed):
        a = {**dict(q=q, sizes=[3], prefix=[16], pages=lens[:1], table=table, lens=lens, max_suffix_len=32), **changed}
        return cache.attend_shared(a.pop("q"), a.pop("sizes"), a.pop("prefix"), a.pop("pages"), a.pop("table"), a.pop("lens"), **a)

    append(), window(), shared()
    for call, bad in [
        (append, dict(k=k.float())), (append, dict(k=k.half())), (append, dict(k=k[:, :1])), (append, dict(v=k[:2])), (append, dict(k=k.cpu())),
        (append, dict(k=k.transpose(0, 1))), (append, dict(slots=slots.int())), (append, dict(slots=slots[:2])), (append, dict(positions=pos.long())),
        (append, dict(positions=pos[:2])), (append, dict(positions=torch.zeros(5, 3, dtype=torch.int32, device="cuda"))),
        (append, dict(cos_sin=turns.half())), (append, dict(cos_sin=turns[:, :40].contiguous())), (append, dict(cos_sin=turns[:, :32])),
        (append, dict(q=q[:2])), (append, dict(q=q, q_out=q[:, :2])), (append, dict(positions=torch.zeros(2, 3, dtype=torch.int32, device="cuda"))),
        (append, dict(axis_of_freq=[0] * 31)),
        (window, dict(q=q.half())), (window, dict(q=q[:, :3])), (window, dict(q=q[..., :32])), (window, dict(q=q[:2])), (window, dict(q_lens=[1, 1])),
        (window, dict(q_lens=[1, 1, 2])), (window, dict(table=table.long())), (window, dict(table=table[:2])), (window, dict(table=table.t())),
        (window, dict(lens=lens.long())), (window, dict(max_kv_len=33)), (window, dict(out=q.float())), (window, dict(out=q[:2])),
        (window, dict(lse=torch.zeros(3, 2, device="cuda"))), (window, dict(scale=0.0)), (window, dict(window=-1)),
        (shared, dict(sizes=[2])), (shared, dict(sizes=[2, 1])), (shared, dict(prefix=[20])), (shared, dict(prefix=[32])), (shared, dict(pages=lens.long())),
        (shared, dict(table=table[:2])), (shared, dict(lens=lens[:2])), (shared, dict(max_suffix_len=33)), (shared, dict(q=q.cpu())),
    ]:
        with pytest.raises(cpkv.CpkvError):
            call(**bad)
    torch.cuda.synchronize()
    assert int(cache.d_status) == 0


def test_example_of_a_serving_step():
    """Compose, append and both attentions together, as examples/serving_step.py runs them."""
    path = pathlib.Path(__file__).parents[1] / "examples" / "serving_step.py"
    spec = importlib.util.spec_from_file_location("serving_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.run()
    assert not any(got["status"])
    assert torch.equal(got["prefill"], got["paged"])
    u = model.bound_of(BF16)
    for a, b in zip(got["decode"], got["window"]):  # the same sums in another order: a step of weights and of the result
        a, b = a.double(), b.double()
        assert bool(((a - b).abs() <= 2 * u * b.abs() + 2 * (u + 2.0**-13) * 5).all())  # weighted |values| below 5
