"""Quantised rows on the GPU: calls that are refused, empty caches, the ends of the number range."""
import numpy as np
import pytest
import torch

import quantised_model as qmodel
import serving_model as model
from paged_kv_cache_compose_gb300 import cpkv
from paged_kv_cache_compose_gb300.cpkv import QuantisedRow
from test_gpu_quantised import cache_of, tensor, turns
from test_gpu_quantised_attend import KIND_NAMES, KINDS, want_window
from test_gpu_serving import page_tables, queries, run_window

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


# --------------------------------------------------------------------------- append: shapes

APPENDS = [cpkv.cpkv_append_quantised, cpkv.cpkv_append_rotary]


def append_inputs(hkv=4, d=64, n=5):
    rng = np.random.default_rng(n)
    pools = qmodel.Pools(2, 16, 1, QuantisedRow.of(hkv, d), BF16)
    wide = tensor(rng.standard_normal((n, 3 * hkv, d)), BF16).cuda()  # a projection's output: strides that any of its slices would pass with
    slots = torch.arange(16, 16 + n).cuda()
    positions, table = torch.arange(n, dtype=torch.int32, device="cuda"), torch.from_numpy(turns(rng, 8, d)).cuda()
    return pools, wide, slots, positions, table


@pytest.mark.parametrize("call", APPENDS, ids=["append_quantised", "append_rotary"])
def test_append_functions_write_what_the_handle_writes(call):
    pools, wide, slots, positions, table = append_inputs()
    one, two = cache_of(pools, BF16), cache_of(pools, BF16)
    q, k, v = wide[:, :4], wide[:, 4:8], wide[:, 8:]
    want = one.append_rotary(k, v, slots, positions, table, q=q)
    q_out = torch.empty_like(want)
    call(k, v, slots, positions, table, table=two.table, d_status=two.d_status, q=q, q_out=q_out)
    assert torch.equal(q_out, want) and bool(one.table.pools[0].any()) and torch.equal(one.table.pools[0], two.table.pools[0])
    assert int(one.d_status) == 0 and int(two.d_status) == 0


@pytest.mark.parametrize("call", APPENDS, ids=["append_quantised", "append_rotary"])
def test_append_functions_refuse_other_heads_and_widths(call):
    """Fewer or narrower heads than the cache's rows have are not read past: the call refuses before anything is launched."""
    pools, wide, slots, positions, table = append_inputs()
    cache = cache_of(pools, BF16)
    k, v = wide[:, 4:8], wide[:, 8:]
    narrow = wide[:, :, :32].contiguous()
    for bad_k, bad_v in [(k[:, :1], v[:, :1]), (k[:, 3:], v[:, 3:]), (wide[:, :5], wide[:, 5:10]), (k, v[:, :3]), (k[:, :3], v),
                         (narrow[:, :4], v), (k, narrow[:, :4]), (narrow[:, :4], narrow[:, :4]),
                         (wide.flatten(1).unflatten(1, (6, 128))[:, :4], v), (k, wide.flatten(1).unflatten(1, (6, 128))[:, :4])]:
        with pytest.raises(cpkv.CpkvError):
            call(bad_k, bad_v, slots, positions, table, table=cache.table, d_status=cache.d_status)
        with pytest.raises(cpkv.CpkvError):
            cache.append_rotary(bad_k, bad_v, slots, positions, table)
    torch.cuda.synchronize()
    assert not bool(cache.table.pools[0].any()) and int(cache.d_status) == 0


# --------------------------------------------------------------------------- attention: no keys

@pytest.mark.parametrize("q_lens, heads", [([1024], 32), ([300] * 3, 16), ([0, 900], 8)], ids=str)
def test_many_query_rows_without_any_keys(q_lens, heads):
    """As over rows of 16 bits: zeros and a log-sum-exp of -infinity, also in a graph."""
    hkv, d = heads // 4, 128
    cache = cache_of(qmodel.Pools(3, 16, 1, QuantisedRow.of(hkv, d), BF16).fill(np.random.default_rng(0)), BF16)
    q = torch.ones(sum(q_lens), heads, d, dtype=BF16, device="cuda")
    lens = torch.zeros(len(q_lens), dtype=torch.int32, device="cuda")
    for pages, most in ((0, 0), (1, 0), (1, 16)):
        out, lse = torch.full_like(q, 7.0), torch.zeros(q.shape[:2], device="cuda")
        table = torch.full((len(q_lens), pages), -7, dtype=torch.int32, device="cuda")

        def attend():
            cache.attend_window(q, q_lens, table, lens, max_kv_len=most, window=3, sinks=2, out=out, lse=lse)

        attend()
        torch.cuda.synchronize()
        assert int(cache.d_status) == 0 and bool((out == 0).all()) and bool(torch.isneginf(lse).all())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            attend()
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert int(cache.d_status) == 0 and bool((out == 0).all())


# --------------------------------------------------------------------------- attention: values near the smallest numbers

def window_of_sizes(nq, hq, kv, sizes, d=64, ps=16):
    """A bf16 cache whose values have these powers of two, one drawn for each token: (case, pools, lists, q)."""
    rng = np.random.default_rng(kv[0] + nq)
    lists, n_pages = page_tables(rng, kv, ps)
    pools = qmodel.Pools(n_pages, ps, 2, QuantisedRow.of(1, d), BF16)
    for page in lists[0]:
        for off in range(ps):
            v = rng.standard_normal((1, d))
            v[0, rng.integers(d)] = 1.75  # the largest of its group, which is therefore not below 2^size
            pools.put(int(page), off, rng.standard_normal((1, d)), np.clip(v, -1.75, 1.75) * 2.0 ** rng.integers(*sizes))
    return (hq, 1, d, ps, 2, BF16, 0, 0, [nq], kv), pools, lists, queries(rng, nq, hq, d, BF16)


def check_scaled(out, lse, want, power):
    """serving_model.check in units of 2^-power, in which its 2^-24 is half a step of bf16's smallest numbers (2^-134) or more."""
    model.check(out.double() * 2.0**power, lse, (want[0] * 2.0**power, want[1], want[2] * 2.0**power), BF16)


# Values of 2^-116 and more have scales of 2^-124, and all of e4m3's multiples of those are bf16 numbers, so each pass's bound is the usual one.
@pytest.mark.parametrize("sizes", [(-116, -110), (-116, -60)], ids=["tiny", "spread"])
@pytest.mark.parametrize("nq, hq, kv", KINDS + [(1, 12, [3000])], ids=KIND_NAMES + ["split-16-rows"])
def test_tiny_values_are_not_lost(nq, hq, kv, sizes):
    case, pools, lists, q = window_of_sizes(nq, hq, kv, sizes)
    out, lse = run_window(cache_of(pools, BF16), case, q, lists)
    want = want_window(case, pools, lists, q)
    assert bool((want[0].abs() > 2.0**-124).any()) and bool(out.any())
    check_scaled(out, lse, want, 110)


@pytest.mark.parametrize("nq, hq, kv", [(1, 2, [3000]), (3, 2, [3000]), (1, 2, [200]), (1, 12, [3000])], ids=["split", "split-queries", "few-keys", "split-16-rows"])
def test_values_of_the_smallest_scale(nq, hq, kv):
    """Scales of 2^-126, the least that the append writes: beside few query rows the values are e4m3 numbers until the end."""
    case, pools, lists, q = window_of_sizes(nq, hq, kv, (-124, -117))
    out, lse = run_window(cache_of(pools, BF16), case, q, lists)
    check_scaled(out, lse, want_window(case, pools, lists, q), 110)


def test_shared_keeps_tiny_values():
    """Of few rows: prefix and suffixes in one split pass."""
    d, ps, sizes, prefix, suffix = 64, 16, [3], [160], [40, 0, 77]
    rng = np.random.default_rng(5)
    lists, n_pages = page_tables(rng, prefix + suffix, ps)
    pools = qmodel.Pools(n_pages, ps, 2, QuantisedRow.of(1, d), BF16)
    for page in range(1, n_pages + 1):
        for off in range(ps):
            pools.put(page, off, rng.standard_normal((1, d)), np.clip(rng.standard_normal((1, d)), -1.75, 1.75) * 2.0**-113)
    q = queries(rng, 3, 4, d, BF16)
    pages, table = lists[0, :10].astype(np.int32), lists[1:]
    lse = torch.empty(3, 4, device="cuda")
    out = cache_of(pools, BF16).attend_shared(q.cuda(), sizes, prefix, torch.from_numpy(pages).cuda(), torch.from_numpy(table).cuda(),
                                              torch.tensor(suffix, dtype=torch.int32).cuda(), max_suffix_len=77, lse=lse)
    check_scaled(out, lse, model.shared(q, sizes, prefix, pages, table, suffix, qmodel.Dense(pools), kv_heads=1, dim=d, scale=d**-0.5), 110)
