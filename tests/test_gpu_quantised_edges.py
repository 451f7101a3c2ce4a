"""Quantised rows on the GPU: calls that are refused, empty caches, the ends of the number range."""
import numpy as np
import pytest
import torch

import quantised_model as qmodel
from paged_kv_cache_compose_gb300 import cpkv
from paged_kv_cache_compose_gb300.cpkv import QuantisedRow
from test_gpu_quantised import cache_of, tensor, turns

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
