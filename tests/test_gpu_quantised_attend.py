"""Attention over quantised rows on the GPU against plain 64-bit implementations on the numbers that the rows hold."""
import importlib.util
import pathlib

import numpy as np
import pytest
import torch

import quantised_model as qmodel
import serving_model as model
from paged_kv_cache_compose_gb300 import cpkv
from paged_kv_cache_compose_gb300.cpkv import QuantisedRow
from paged_kv_cache_compose_gb300.runtime import PagedCache, QuantisedCache
from test_gpu_quantised import cache_of
from test_gpu_serving import BF16, FP16, MIXED, SHARED, WINDOW, page_tables, queries, run_window
from test_gpu_serving_edges import workspace_at

pytestmark = pytest.mark.gpu


def name(case):
    return "-".join(str(x).replace(" ", "") for x in case)[:80]


def window_case(case, seed=0, width=None):
    hq, hkv, d, ps, cp, dtype, w, sinks, q_lens, kv_lens = case
    rng = np.random.default_rng(seed + sum(kv_lens))
    table, n_pages = page_tables(rng, kv_lens, ps)
    pools = qmodel.Pools(n_pages, ps, cp, QuantisedRow.of(hkv, d), dtype, width).fill(rng)
    return rng, pools, table, queries(rng, sum(q_lens), hq, d, dtype)


def want_window(case, pools, table, q):
    hq, hkv, d, ps, cp, dtype, w, sinks, q_lens, kv_lens = case
    return model.window(q, q_lens, table, kv_lens, qmodel.Dense(pools), kv_heads=hkv, dim=d, window=w, sinks=sinks, scale=d**-0.5)


MORE = [
    (20, 1, 64, 16, 2, FP16, 0, 0, [1, 1], [700, 64]),  # several row tiles of one token
    (160, 1, 64, 48, 2, BF16, 0, 0, [1], [1500]),
    (300, 1, 128, 32, 2, BF16, 90, 7, [1, 2], [1030, 400]),  # more heads than an item has rows
    (12, 1, 128, 128, 2, BF16, 0, 0, [11], [4000]),  # few rows over long keys: parts of two streams
    (4, 1, 64, 16, 12, FP16, 0, 0, [40], [600]),
    (3, 3, 64, 1, 2, BF16, 0, 0, [1, 1, 1], [3000, 5, 1700]),  # an odd number of heads, lines of units
    (24, 3, 128, 16, 2, FP16, 700, 9, [2, 2], [2900, 1500]),
    # row tiles enough that the rows are read back first
    (8, 1, 64, 16, 2, BF16, 0, 0, [200], [333]),
    (8, 1, 128, 1, 3, FP16, 0, 0, [400, 10], [431, 200]),
    (16, 2, 128, 64, 2, BF16, 150, 40, [300, 0, 230], [700, 90, 220]),  # one request shorter than its queries
    (5, 1, 64, 24, 2, FP16, 33, 0, [700], [1500]),
]


@pytest.mark.parametrize("case", WINDOW + MORE, ids=name)
def test_window_matches_64_bits(case):
    hkv, d, ps, dtype = case[1], case[2], case[3], case[5]
    _, pools, table, q = window_case(case)
    cache = cache_of(pools, dtype)
    out, lse = run_window(cache, case, q, table)
    assert int(cache.d_status) == 0
    model.check(out, lse, want_window(case, pools, table, q), dtype)
    again, lse2 = run_window(cache, case, q, table)
    assert torch.equal(out, again) and torch.equal(lse, lse2)  # the same bits every time


@pytest.mark.parametrize("case", [c for c in WINDOW + MORE if c[6]], ids=name)
def test_window_reads_nothing_that_no_query_sees(case):
    """Rows behind the window and past the length hold no numbers, scales neither, and pages wholly there have no page id."""
    hq, hkv, d, ps, cp, dtype, w, sinks, q_lens, kv_lens = case
    _, pools, table, q = window_case(case)
    want, want_lse = run_window(cache_of(pools, dtype), case, q, table)
    for b, (nq, kv) in enumerate(zip(q_lens, kv_lens)):
        first = max(0, kv - nq - w + 1)
        for page in range(-(-kv // ps)):
            seen = np.array([nq > 0 and t < kv and (t >= first or t < min(sinks, first)) for t in range(page * ps, page * ps + ps)])
            lp = int(table[b, page])
            pools.slabs[lp % cp][lp // cp][~seen] = 0xFF
            if not seen.any():
                table[b, page] = -5
    poisoned = cache_of(pools, dtype)
    out, lse = run_window(poisoned, case, q, table)
    assert int(poisoned.d_status) == 0
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


@pytest.mark.parametrize("what", ["element", "scale"])
@pytest.mark.parametrize("case", MIXED + [(8, 1, 64, 16, 2, BF16, 0, 0, [200], [333]), (16, 2, 128, 24, 2, FP16, 50, 3, [150, 90], [400, 90])], ids=name)
def test_window_no_numbers_reach_only_the_rows_that_see_them(case, what):
    """Keys and values that are no numbers (an element of them, or their scale) where some query tokens see them and others do not."""
    hq, hkv, d, ps, cp, dtype, w, sinks, q_lens, kv_lens = case
    rng, pools, table, q = window_case(case)
    row = pools.row
    for b, (nq, kv) in enumerate(zip(q_lens, kv_lens)):
        edge = kv - nq - (w or 10**6) + nq // 2
        for j, key in [(kv - 1, False), (kv - nq // 3 - 1, False), (kv - nq // 2, True), (edge, False), (edge + 1, True)]:
            if 0 <= j < kv:
                raw = pools.at(int(table[b, j // ps]), j % ps)
                if what == "element":
                    raw[(row.key_offset if key else row.value_offset) + rng.integers(0, d)] = 0x7F + 128 * (j % 2)
                else:
                    at = row.key_scale_offset if key else row.value_scale_offset
                    raw[at:at + 4] = np.array([np.nan], np.float32).view(np.uint8)
    want = want_window(case, pools, table, q)
    cache = cache_of(pools, dtype)
    out, lse = run_window(cache, case, q, table)
    assert int(cache.d_status) == 0
    finite = want[0].isfinite()
    assert not finite.all()
    assert torch.equal(out.cpu().isfinite(), finite)
    seen = [torch.where(finite, x, 0.0) for x in (out.double().cpu(), want[0], want[2])]
    model.check(seen[0], None, (seen[1], want[1], seen[2]), dtype)
    assert torch.equal(lse.cpu().isnan(), want[1].isnan())


KINDS = [(1, 2, [3000]), (3, 2, [3000]), (1, 2, [200]), (64, 1, [3000]), (300, 1, [900]), (400, 4, [500])]
KIND_NAMES = ["split", "split-queries", "few-keys", "parts", "tile", "unpacked"]


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("nq, hq, kv", KINDS, ids=KIND_NAMES)
def test_many_small_weights_beside_one_large(nq, hq, kv, dtype):
    """One key's weight is 2^26 times the others', whose values are all that the result is made of; its own are zeros, or nearly."""
    d, ps = 64, 16
    for own in (0.0, 2.0**-10):
        rng = np.random.default_rng(kv[0])
        lists, n_pages = page_tables(rng, kv, ps)
        pools = qmodel.Pools(n_pages, ps, 2, QuantisedRow.of(1, d), dtype)
        for page in lists[0]:
            for off in range(ps):
                pools.put(int(page), off, np.zeros((1, d)), np.ones((1, d)))
        k = np.zeros((1, d))
        k[0, 0] = 9.0  # an e4m3 number: a score of 9 * 16 / 8, a weight of e^18 (2^26)
        pools.put(int(lists[0, 0]), 0, k, np.full((1, d), own))
        q = torch.zeros(nq, hq, d, dtype=dtype)
        q[..., 0] = 16.0
        case = (hq, 1, d, ps, 2, dtype, 0, 0, [nq], kv)
        out, lse = run_window(cache_of(pools, dtype), case, q, lists)
        want = want_window(case, pools, lists, q)
        # Beside more than 16 rows the largest weight is held as 2^7 or more in the type, whose steps in fp16 are 2^-24 below
        # 2^-14: half a step is 2^-32 of the largest weight, for each of kv keys whose values are 1 here.  In units of the
        # bound's steps of `size`, which is the sum of the weights, 2^-26 each:
        more = kv[0] * 2.0**-32 / (2.0**-11 + 2.0**-13) if dtype is FP16 and nq * hq > 16 else 0.0
        model.check(out, lse, (want[0], want[1], want[2] + more), dtype)


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("nq, hq, kv", KINDS, ids=KIND_NAMES)
def test_scales_far_apart(nq, hq, kv, dtype):
    """Values of very different magnitude from token to token (rows of zeros among them), and queries near the type's limits."""
    hkv, d, ps = 1, 64, 16
    rng = np.random.default_rng(kv[0] + 1)
    lists, n_pages = page_tables(rng, kv, ps)
    far = 12 if dtype is FP16 else 90
    pools = qmodel.Pools(n_pages, ps, 2, QuantisedRow.of(hkv, d), dtype)
    for page in lists[0]:
        for off in range(ps):
            size = 2.0 ** rng.integers(-far, 4) * (rng.random() > 0.2)
            pools.put(int(page), off, rng.standard_normal((1, d)) * 2.0 ** -far, rng.standard_normal((1, d)) * size)
    q = queries(rng, nq, hq, d, dtype, 1.5 * 2.0**far)
    q[..., 3] *= 2.0**-far  # small elements beside large ones
    case = (hq, hkv, d, ps, 2, dtype, 0, 0, [nq], kv)
    want = want_window(case, pools, lists, q)
    out, lse = run_window(cache_of(pools, dtype), case, q, lists)
    model.check(out, lse, want, dtype)


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("nq, hq, kv", KINDS, ids=KIND_NAMES)
def test_scales_that_no_append_writes(nq, hq, kv, dtype):
    hkv, d, ps = 1, 128, 16
    case = (hq, hkv, d, ps, 2, dtype, 0, 0, [nq], kv)
    rng, pools, lists, q = window_case(case)
    row = pools.row
    for slab in pools.slabs:
        for at in (row.key_scale_offset, row.value_scale_offset):
            slab[..., at:at + 4] = rng.uniform(0.001, 0.01, slab.shape[:2] + (1,)).astype(np.float32).view(np.uint8).reshape(*slab.shape[:2], 4)
    out, lse = run_window(cache_of(pools, dtype), case, q, lists)
    want = want_window(case, pools, lists, q)
    # beside more than 16 rows keys and values are rounded to the type: scores off by u |q|.|k| scale, weights by twice
    # their factor, values by u
    u = model.bound_of(dtype)
    k = np.concatenate([pools.rows(slab.reshape(-1, slab.shape[-1]))[0][:, 0] for slab in pools.slabs])
    score = u * float((q.double().abs().numpy().reshape(-1, d) @ np.abs(k).T).max()) * d**-0.5
    assert score < 0.25
    rel = 2.0**-13 + 2 * u + (np.exp(2 * score) - 1 if nq * hq > 16 else 0.0)
    assert bool(((out.double().cpu() - want[0]).abs() <= u * want[0].abs() + rel * want[2] + 2.0**-24).all())
    assert float((lse.double().cpu() - want[1]).abs().max()) <= 2.0**-13 + (score if nq * hq > 16 else 0.0)


@pytest.mark.parametrize("nq", [1, 3, 50])
def test_window_reports_bad_pages_and_lengths(nq):
    """A bad page id reads as zero rows, a length past the bound is clamped; both raise their bit."""
    case = (4, 1, 64, 16, 2, BF16, 0, 0, [nq, nq], [100, 60])
    rng, pools, table, q = window_case(case)
    good = table.copy()
    for bad in (-1, 0, 1 << 29):
        table[0, 2] = bad
        cache = cache_of(pools, BF16)
        out, lse = run_window(cache, case, q, table)
        assert int(cache.d_status) == cpkv.STATUS_PAGE_OOB
        zeroed = qmodel.Pools(1, 16, 2, pools.row, BF16)
        zeroed.slabs = [s.copy() for s in pools.slabs]
        lp = int(good[0, 2])
        zeroed.slabs[lp % 2][lp // 2] = 0
        model.check(out, lse, want_window(case, zeroed, good, q), BF16)
    cache = cache_of(pools, BF16)
    out, lse = run_window(cache, case, q, good, max_kv=90)
    assert int(cache.d_status) == cpkv.STATUS_OUT_CAPACITY
    model.check(out, lse, want_window(case[:9] + ([90, 60],), pools, good, q), BF16)
    cache = cache_of(pools, BF16)
    out = cache.attend_window(q.cuda(), [nq, nq], torch.from_numpy(good).cuda(), torch.tensor([-3, 60], dtype=torch.int32).cuda(), max_kv_len=100)
    assert int(cache.d_status) == cpkv.STATUS_OUT_CAPACITY and bool((out[:nq] == 0).all())


@pytest.mark.parametrize("nq", [1, 33])
def test_window_strides_layouts_and_dense_pages(nq):
    """Queries and outputs as slices, rows in another order with room between, one dense buffer whose page 0 counts."""
    rng = np.random.default_rng(9)
    hq, hkv, d, ps, kv = 6, 2, 64, 16, 150
    row = QuantisedRow(336, 160, 16, 4, 296, hkv, d, d, 0)  # key scales before the values, which are before the keys
    pools = qmodel.Pools(9, ps, 1, row, BF16).fill(rng)
    table = np.arange(10, dtype=np.int32)[None]
    wide = queries(rng, nq, hq + 4, d, BF16).cuda()
    holder = torch.zeros(nq, hq + 1, d, dtype=BF16, device="cuda")
    cache = cache_of(pools, BF16, dense=True)
    lse = torch.empty(nq, hq, device="cuda")
    q = wide[:, 2:2 + hq]
    out = cache.attend_window(q, [nq], torch.from_numpy(table).cuda(), torch.tensor([kv], dtype=torch.int32).cuda(),
                              max_kv_len=kv, window=70, sinks=3, scale=0.3, out=holder[:, :hq], lse=lse)
    assert int(cache.d_status) == 0 and bool((holder[:, hq] == 0).all())
    want = model.window(q.cpu(), [nq], table, [kv], qmodel.Dense(pools), kv_heads=hkv, dim=d, window=70, sinks=3, scale=0.3)
    model.check(out, lse, want, BF16)


@pytest.mark.parametrize("q_lens, heads", [([1, 1], 4), ([1] * 60, 4), ([2, 0, 3], 4), ([40, 300], 4)], ids=["few-keys", "line", "queries", "tile"])
def test_requests_without_any_keys(q_lens, heads):
    hkv, d = 4, 64
    pools = qmodel.Pools(3, 16, 1, QuantisedRow.of(hkv, d), BF16).fill(np.random.default_rng(0))
    cache = cache_of(pools, BF16)
    q = torch.ones(sum(q_lens), heads, d, dtype=BF16, device="cuda")
    lse = torch.zeros(q.shape[:2], device="cuda")
    for pages, most in ((0, 0), (1, 16)):
        out = cache.attend_window(q, q_lens, torch.full((len(q_lens), pages), -7, dtype=torch.int32, device="cuda"),
                                  torch.zeros(len(q_lens), dtype=torch.int32, device="cuda"), max_kv_len=most, lse=lse.zero_(), window=3, sinks=2)
        torch.cuda.synchronize()
        assert int(cache.d_status) == 0 and bool((out == 0).all()) and bool(torch.isneginf(lse).all())


# --------------------------------------------------------------------------- shared

@pytest.mark.parametrize("case", SHARED + [
    (48, 1, 64, 16, 2, FP16, [3, 1], [208, 64], [40, 3, 1, 90]),
    (160, 1, 64, 16, 2, BF16, [2], [400], [5, 200]),
    (300, 1, 128, 32, 2, BF16, [1, 1], [96, 1024], [70, 1]),
    (8, 1, 128, 1, 3, FP16, [24], [700], [1 + 11 * i for i in range(24)]),
    (16, 1, 128, 16, 2, BF16, [1], [3008], [2000]),
    # prefixes of many rows, whose requests' suffixes are of few
    (16, 2, 64, 16, 2, BF16, [5, 0, 20], [96, 32, 0], [0, 1, 64, 65, 200] + [(37 * i) % 130 for i in range(20)]),
    (32, 2, 128, 8, 3, FP16, [3] * 17, [8 * i for i in range(17)], [(7 * i) % 90 for i in range(51)]),
    (24, 8, 64, 64, 1, BF16, [60], [4160], [1000 - 16 * i for i in range(60)]),
    (8, 1, 128, 16, 2, BF16, [12], [64], [0] * 12),
], ids=name)
def test_shared_matches_64_bits(case):
    hq, hkv, d, ps, cp, dtype, sizes, prefix, suffix = case
    rng = np.random.default_rng(sum(suffix))
    lists, n_pages = page_tables(rng, prefix + suffix, ps)
    pools = qmodel.Pools(n_pages, ps, cp, QuantisedRow.of(hkv, d), dtype).fill(rng)
    prefix_pages = np.concatenate([lists[g, :n // ps] for g, n in enumerate(prefix)]).astype(np.int32)
    table = lists[len(prefix):]
    q = queries(rng, sum(sizes), hq, d, dtype)
    want = model.shared(q, sizes, prefix, prefix_pages, table, suffix, qmodel.Dense(pools), kv_heads=hkv, dim=d, scale=d**-0.5)
    cache = cache_of(pools, dtype)
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


def test_shared_of_two_passes_in_a_graph():
    """Prefix and suffixes by two kernels and joined, captured: replays follow the lengths and agree with a plain call."""
    rng = np.random.default_rng(11)
    hq, hkv, d, ps, n = 16, 2, 64, 16, 40
    lists, n_pages = page_tables(rng, [640] + [300] * n, ps)
    pools = qmodel.Pools(n_pages, ps, 2, QuantisedRow.of(hkv, d), BF16).fill(rng)
    cache = cache_of(pools, BF16)
    q = queries(rng, n, hq, d, BF16).cuda()
    prefix_pages, table = torch.from_numpy(lists[0, :40].astype(np.int32)).cuda(), torch.from_numpy(lists[1:]).cuda()
    lens = torch.ones(n, dtype=torch.int32).cuda()

    def attend(**more):
        return cache.attend_shared(q, [n], [640], prefix_pages, table, lens, max_suffix_len=300, **more)

    attend()
    torch.cuda.synchronize()
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(q)
    with torch.cuda.graph(graph):
        attend(out=out)
    for _ in range(3):
        suffix = rng.integers(0, 301, n).astype(np.int32)
        lens.copy_(torch.from_numpy(suffix))
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, attend())
        want = model.shared(q.cpu(), [n], [640], prefix_pages.cpu().numpy(), lists[1:], suffix.tolist(), qmodel.Dense(pools),
                            kv_heads=hkv, dim=d, scale=d**-0.5)
        lse = torch.empty(n, hq, device="cuda")
        model.check(attend(lse=lse), lse, want, BF16)
    assert int(cache.d_status) == 0


def test_shared_takes_its_workspace_and_no_less():
    rng = np.random.default_rng(12)
    hq, hkv, d, ps, n = 8, 1, 128, 16, 24
    lists, n_pages = page_tables(rng, [160] + [40] * n, ps)
    pools = qmodel.Pools(n_pages, ps, 2, QuantisedRow.of(hkv, d), FP16).fill(rng)
    cache = cache_of(pools, FP16)
    q = queries(rng, n, hq, d, FP16).cuda()
    need = cpkv.cpkv_attend_shared_quantised_workspace_bytes(n, hq, hkv, d, [n], [160], 40)
    args = (q, [n], [160], torch.from_numpy(lists[0, :10].astype(np.int32)).cuda(), torch.from_numpy(lists[1:]).cuda(),
            torch.arange(1, n + 1, dtype=torch.int32).cuda())
    room = torch.full((need + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    at = -room.data_ptr() % 16
    out = cache.attend_shared(*args, max_suffix_len=40, workspace=room[at:at + need])
    assert torch.equal(out, cache.attend_shared(*args, max_suffix_len=40))
    assert (room[at + need:] == 0x5A).all() and (room[:at] == 0x5A).all()
    with pytest.raises(cpkv.CpkvError) as e:
        cache.attend_shared(*args, max_suffix_len=40, workspace=room[at:at + need - 16])
    assert e.value.code == cpkv.CPKV_ERR_CAPACITY


def test_shared_reports_bad_pages():
    rng = np.random.default_rng(3)
    pools = qmodel.Pools(20, 16, 2, QuantisedRow.of(1, 64), BF16).fill(rng)
    q = queries(rng, 40, 2, 64, BF16).cuda()
    for n in (2, 40):
        cache = cache_of(pools, BF16)
        lens, table = torch.full((n,), 3, dtype=torch.int32).cuda(), torch.full((n, 1), 5, dtype=torch.int32).cuda()
        for prefix_pages in ([1, 1000], [0, 2], [-1, 2]):
            cache.d_status.zero_()
            cache.attend_shared(q[:n], [n], [32], torch.tensor(prefix_pages, dtype=torch.int32).cuda(), table, lens, max_suffix_len=16)
            assert int(cache.d_status) == cpkv.STATUS_PAGE_OOB


# --------------------------------------------------------------------------- graphs, workspaces, waits, refusals

@pytest.mark.parametrize("tokens", [1, 24, 260], ids=["split", "tile", "unpacked"])
def test_in_a_graph_on_another_stream_follows_the_lengths(tokens):
    case = (8, 2, 128, 16, 2, BF16, 100, 4, [tokens] * 3, [300, 290, 280])
    rng, pools, table, q = window_case(case)
    cache = cache_of(pools, BF16)
    lens = torch.full((3,), tokens, dtype=torch.int32).cuda()
    d_q, d_table = q.cuda(), torch.from_numpy(table).cuda()
    out, lse = torch.empty_like(d_q), torch.empty(3 * tokens, 8, device="cuda")

    def step():
        cache.attend_window(d_q, [tokens] * 3, d_table, lens, max_kv_len=300, window=100, sinks=4, out=out, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for now in ([300, 90, 200], [tokens + 5, 0, 104]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        model.check(out, lse, want_window(case[:9] + (now,), pools, table, q), BF16, str(now))
    assert int(cache.d_status) == 0


@pytest.mark.parametrize("offset", [0, 16, 48])
@pytest.mark.parametrize("q_lens, kv_lens", [([11], [4000]), ([1, 1], [3000, 900]), ([140], [900])], ids=["tile", "split", "unpacked"])
def test_workspace_at_any_multiple_of_16(q_lens, kv_lens, offset):
    """The workspace that the sizing call asks for, wherever it begins, is enough and all that is written."""
    case = (12, 1, 128, 64, 2, BF16, 0, 0, q_lens, kv_lens)
    _, pools, lists, q = window_case(case)
    cache = cache_of(pools, BF16)
    need = cpkv.cpkv_attend_window_quantised_workspace_bytes(len(q_lens), 12, 1, 128, q_lens, max(kv_lens))
    workspace, untouched = workspace_at(need, offset)
    d_q = q.cuda()
    out, lse = torch.empty_like(d_q), torch.empty(q.shape[:2], device="cuda")
    cpkv.cpkv_attend_window_quantised(d_q, q_lens, torch.from_numpy(lists).cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda(),
                                      table=cache.table, max_kv_len=max(kv_lens), window=0, sinks=0, scale=128**-0.5, out=out, lse=lse,
                                      workspace=workspace, d_status=cache.d_status)
    torch.cuda.synchronize()
    assert int(cache.d_status) == 0 and untouched()
    model.check(out, lse, want_window(case, pools, lists, q), BF16)
    with pytest.raises(cpkv.CpkvError):
        cpkv.cpkv_attend_window_quantised(d_q, q_lens, torch.from_numpy(lists).cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda(),
                                          table=cache.table, max_kv_len=max(kv_lens), window=0, sinks=0, scale=0.1, out=out, lse=lse,
                                          workspace=workspace[:-16], d_status=cache.d_status)


def test_long_cache_offsets_past_32_bits():
    """Pages beyond 4 GB of one pool: read, attended to, written."""
    ps, hkv, d = 64, 8, 128
    row = QuantisedRow.of(hkv, d)
    pages = (5 << 30) // (ps * row.row_bytes)
    pool = torch.zeros(pages, ps, row.row_bytes, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(4)
    small = qmodel.Pools(2, ps, 1, row, BF16).fill(rng)
    pool[-2:] = torch.from_numpy(small.slabs[0][1:]).cuda()
    cache = QuantisedCache([pool], page_size=ps, kv_heads=hkv, key_dim=d)
    table = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32).cuda()
    for nq in (1, 40):
        q = queries(rng, nq, hkv, d, BF16)
        lse = torch.empty(nq, hkv, device="cuda")
        out = cache.attend_window(q.cuda(), [nq], table, torch.tensor([100], dtype=torch.int32).cuda(), max_kv_len=128, lse=lse)
        want = model.window(q, [nq], [[1, 2]], [100], qmodel.Dense(small), kv_heads=hkv, dim=d, window=0, sinks=0, scale=d**-0.5)
        model.check(out, lse, want, BF16)
    slot = torch.tensor([(pages - 1) * ps + 5]).cuda()
    k, v = cache.read_rows(slot)
    ref = small.rows(small.at(2, 5)[None])
    assert np.array_equal(k.double().cpu().numpy(), ref[0]) and np.array_equal(v.double().cpu().numpy(), ref[1])
    cache.append_rotary(v, k, slot, torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cat([torch.ones(1, 64), torch.zeros(1, 64)], 1).cuda())
    again = cache.read_rows(slot)
    assert torch.equal(again[0], v) and torch.equal(again[1], k) and int(cache.d_status) == 0


@pytest.mark.parametrize("d, tokens", [(64, 64), (128, 64), (128, 2048)])
def test_blocks_that_give_up_leave_the_gpu_usable(d, tokens):
    pages = 1024
    rows = torch.zeros(pages, 64, 2 * d + 16, dtype=torch.uint8, device="cuda")
    table, lens = torch.arange(pages, dtype=torch.int32, device="cuda"), torch.tensor([64 * pages], dtype=torch.int32, device="cuda")
    q = torch.zeros(tokens, d, dtype=BF16, device="cuda")
    out = torch.empty_like(q)
    case = (8, 2, d, 16, 2, BF16, 0, 0, [24], [500])
    _, pools, lists, small = window_case(case)
    want = want_window(case, pools, lists, small)
    for wait_ns in (0, 1000, 10_000, 50_000, 10**9):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        cpkv.cpkv_selftest_attend_quantised_timeout(rows, table, lens, q, out, wait_ns, status)
        torch.cuda.synchronize()
        # 65536 keys take hundreds of us: no block gets through without a wait of 50; none of them waits for a second
        assert int(status) == (0 if wait_ns == 10**9 else cpkv.STATUS_TIMEOUT), wait_ns
        assert wait_ns < 10**9 or bool((out == 0).all())
        cache = cache_of(pools, BF16)
        model.check(*run_window(cache, case, small, lists), want, BF16)
        assert int(cache.d_status) == 0


def test_calls_refuse_what_their_tensors_cannot_be():
    d, ps = 64, 16
    row = QuantisedRow.of(2, d)
    cache = QuantisedCache([torch.zeros(4, ps, row.row_bytes, dtype=torch.uint8, device="cuda")], page_size=ps, kv_heads=2, key_dim=d)
    latent = QuantisedCache([torch.zeros(4, ps, 656, dtype=torch.uint8, device="cuda")], page_size=ps, kv_heads=1, key_dim=64, value_dim=512, keep_keys=True)
    kept = QuantisedCache([torch.zeros(4, ps, 656, dtype=torch.uint8, device="cuda")], page_size=ps, kv_heads=1, key_dim=64, keep_keys=True)
    q = torch.zeros(3, 4, d, dtype=BF16, device="cuda")
    table, lens = torch.ones(3, 2, dtype=torch.int32, device="cuda"), torch.ones(3, dtype=torch.int32, device="cuda")

    def window(cache=cache, q=q, **changed):
        return cache.attend_window(q, None, table, lens, max_kv_len=32, **changed)

    def shared(cache=cache, q=q, **changed):
        return cache.attend_shared(q, [3], [16], lens[:1], table, lens, max_suffix_len=32, **changed)

    for call in (window, shared):
        call()
        for bad in (dict(q=q.half()), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(cache=latent), dict(cache=kept), dict(out=q[:2]), dict(scale=0.0),
                    dict(lse=torch.zeros(3, 2, device="cuda")), dict(workspace=torch.zeros(16, dtype=torch.uint8))):
            with pytest.raises(cpkv.CpkvError):
                call(**bad)
    torch.cuda.synchronize()
    assert int(cache.d_status) == 0 and int(latent.d_status) == 0


# --------------------------------------------------------------------------- together

def test_a_serving_run_on_quantised_rows():
    """A prompt appended, read back and attended to as a dense prefill; then decode steps with and without sharing it."""
    rng = np.random.default_rng(12)
    hq, hkv, d, ps, cp, prompt, b, steps = 8, 2, 64, 16, 2, 96, 5, 3
    row = QuantisedRow.of(hkv, d)
    pages = prompt // ps + b
    order = 1 + rng.permutation(pages)
    pools = qmodel.Pools(pages, ps, cp, row, BF16)
    cache = cache_of(pools, BF16)
    turns = torch.from_numpy(np.concatenate([np.cos(a := np.arange(200)[:, None] * 10.0 ** (-np.arange(d // 2) / 8)), np.sin(a)], 1).astype(np.float32)).cuda()

    def heads(n, h):
        return queries(rng, n, h, d, BF16, 1.0).cuda()

    slots = torch.from_numpy(np.concatenate([order[i] * ps + np.arange(ps) for i in range(prompt // ps)])).cuda()
    q, k, v = heads(prompt, hq), heads(prompt, hkv), heads(prompt, hkv)
    q = cache.append_rotary(k, v, slots, torch.arange(prompt, dtype=torch.int32, device="cuda"), turns, q=q)
    d_prompt = torch.from_numpy(order[:prompt // ps].astype(np.int32)).cuda()
    n = torch.tensor([prompt], dtype=torch.int32, device="cuda")
    over_quantised = cache.attend_window(q, [prompt], d_prompt[None], n, max_kv_len=prompt)
    # read back: the same prefill over plain rows.  Both are of the same numbers, weighed in fp16 and in bf16: each lies
    # within the bound of its own roundings around the value in 64 bits
    dense = torch.zeros(prompt, 2 * hkv * d, dtype=BF16, device="cuda")
    cache.read_rows(slots, k_out=dense[:, :hkv * d].unflatten(1, (hkv, d)), v_out=dense[:, hkv * d:].unflatten(1, (hkv, d)))
    plain = PagedCache([dense.view(-1, ps, 2 * hkv * d)], page_size=ps, kv_heads=hkv, key_dim=d, dense=True)
    over_plain = plain.attend_window(q, [prompt], torch.arange(prompt // ps, dtype=torch.int32, device="cuda")[None], n, max_kv_len=prompt)
    pools.slabs = [t.cpu().numpy() for t in cache.table.pools]
    want = model.window(q.cpu(), [prompt], d_prompt[None].cpu().numpy(), [prompt], qmodel.Dense(pools), kv_heads=hkv, dim=d, window=0, sinks=0, scale=d**-0.5)
    for got in (over_quantised, over_plain):
        model.check(got, None, want, BF16)

    own = torch.from_numpy(order[prompt // ps:].astype(np.int32)).cuda()[:, None]
    both = torch.cat([d_prompt.expand(b, -1), own], 1)
    for step in range(steps):
        q1, k1, v1 = heads(b, hq), heads(b, hkv), heads(b, hkv)
        positions = torch.full((b,), prompt + step, dtype=torch.int32, device="cuda")
        q1 = cache.append_rotary(k1, v1, own[:, 0].long() * ps + step, positions, turns, q=q1)
        suffix = torch.full((b,), step + 1, dtype=torch.int32, device="cuda")
        one = cache.attend_shared(q1, [b], [prompt], d_prompt, own, suffix, max_suffix_len=ps)
        two = cache.attend_window(q1, None, both, prompt + suffix, max_kv_len=prompt + ps)
        pools.slabs = [t.cpu().numpy() for t in cache.table.pools]
        want = model.window(q1.cpu(), [1] * b, both.cpu().numpy(), [prompt + step + 1] * b, qmodel.Dense(pools), kv_heads=hkv, dim=d, window=0, sinks=0,
                            scale=d**-0.5)
        model.check(one, None, want, BF16)
        model.check(two, None, want, BF16)
    assert int(cache.d_status) == 0 and int(plain.d_status) == 0


def test_example_of_a_serving_step_on_quantised_rows():
    """Compose, append and both attentions together on quantised rows, as examples/serving_step.py runs them."""
    path = pathlib.Path(__file__).parents[1] / "examples" / "serving_step.py"
    spec = importlib.util.spec_from_file_location("serving_step", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    got = example.run(quantised=True)
    assert not any(got["status"])
    assert torch.equal(got["prefill"], got["paged"])
    u = model.bound_of(BF16)
    for a, b in zip(got["decode"], got["window"]):  # each within its own bound: a step of weights and of the result
        a, b = a.double(), b.double()
        assert bool(((a - b).abs() <= 2 * u * b.abs() + 2 * (u + 2.0**-13) * 5).all())  # weighted |values| below 5
