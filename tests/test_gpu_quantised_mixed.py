"""Quantised prefixes of many rows by the tile pass beside their requests' suffixes by the split pass, one joined result.

The two passes are taken where the suffixes come to two key tiles of 128 for each SM; each case here is checked to have the
workspace of that form, which holds the parts of both passes, and not that of the single pass."""
import numpy as np
import pytest
import torch

import quantised_model as qmodel
import serving_model as model
from paged_kv_cache_compose_gb300 import cpkv
from paged_kv_cache_compose_gb300.cpkv import QuantisedRow
from test_gpu_quantised import cache_of
from test_gpu_quantised_edges import check_scaled
from test_gpu_serving import page_tables, queries
from test_gpu_serving_edges import workspace_at

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


def up(n, to):
    return -(-n // to) * to


def two_passes(n, hq, hkv, d, sizes, prefix, most):
    """Whether a call runs as two passes: by its suffixes' key tiles, and by its workspace."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = n * hkv * -(-most // 128)
    need = cpkv.cpkv_attend_shared_quantised_workspace_bytes(n, hq, hkv, d, sizes, prefix, most)
    # the split pass's part of it: two slots a block, one a request and head, of 16 rows
    blocks = hkv * min(1024 // hkv, n * -(-most // 64))
    slots = (2 * blocks + n * hkv) * 16
    split = up((n + 1) * 4, 256) + up(slots * 8, 256) + up(slots * d * 4, 256)
    return tiles >= 2 * sms and need > split and need != cpkv.cpkv_attend_shared_workspace_bytes(n, hq, hkv, d, sizes, prefix, most), need


class Call:
    """A shared call over random rows, and its values in 64 bits for a sample of the requests."""

    def __init__(self, case, seed=0, spare=0):
        hq, hkv, d, ps, cp, dtype, sizes, prefix, suffix = self.case = case
        self.rng = rng = np.random.default_rng(seed + sum(suffix))
        self.most = max(suffix) + spare
        lists, n_pages = page_tables(rng, list(prefix) + [self.most] * len(suffix), ps)
        self.pools = qmodel.Pools(n_pages, ps, cp, QuantisedRow.of(hkv, d), dtype).fill(rng)
        self.prefix_pages = np.concatenate([lists[g, :n // ps] for g, n in enumerate(prefix)]).astype(np.int32)
        self.lists = np.ascontiguousarray(lists[len(prefix):, :-(-self.most // ps)])
        self.q = queries(rng, len(suffix), hq, d, dtype)
        self.suffix = list(suffix)
        two, self.need = two_passes(len(suffix), hq, hkv, d, sizes, prefix, self.most)
        assert two
        self.cache = cache_of(self.pools, dtype)
        self.d_q, self.d_prefix = self.q.cuda(), torch.from_numpy(self.prefix_pages).cuda()
        self.d_table, self.d_lens = torch.from_numpy(self.lists).cuda(), torch.tensor(self.suffix, dtype=torch.int32).cuda()

    def __call__(self, **more):
        hq, hkv, d, ps, cp, dtype, sizes, prefix, _ = self.case
        lse = more.pop("lse", None)
        lse = torch.full((len(self.suffix), hq), 7.0, device="cuda") if lse is None else lse
        out = self.cache.attend_shared(more.pop("q", self.d_q), sizes, prefix, self.d_prefix, self.d_table, self.d_lens, max_suffix_len=self.most, lse=lse, **more)
        return out, lse

    def check(self, out, lse, requests=24, heads=None, rows=None):
        """A sample of the requests, among them the first and last of each group, against 64 bits."""
        hq, hkv, d, ps, cp, dtype, sizes, prefix, _ = self.case
        ends = np.cumsum(sizes)
        chosen = {0, len(self.suffix) - 1} | set(self.rng.permutation(len(self.suffix))[:requests].tolist())
        if len(sizes) <= 20:
            chosen |= {int(e) - 1 for e in ends if e} | {int(e - s) for e, s in zip(ends, sizes) if s}
        chosen = sorted(chosen)
        dense = qmodel.Dense(rows or self.pools)
        p0 = np.concatenate([[0], np.cumsum([n // ps for n in prefix])])
        for g, n in enumerate(sizes):
            mine = [b for b in chosen if ends[g] - n <= b < ends[g]]
            if not mine:
                continue
            want = model.shared(self.q[mine], [len(mine)], [prefix[g]], self.prefix_pages[p0[g]:p0[g + 1]], self.lists[mine], [self.suffix[b] for b in mine],
                                dense, kv_heads=hkv, dim=d, scale=d**-0.5)
            at = torch.tensor(mine)
            model.check(out.cpu()[at], None if lse is None else lse.cpu()[at], want, dtype, f"group {g}")


EMPTY = [0, 1, 63, 64, 65, 127, 128, 129]

CASES = {  # q heads, kv heads, dim, ps, cp, dtype, group sizes, prefix lens, suffix lens
    "bf16-128-4-rows": (32, 8, 128, 64, 8, BF16, [40], [1024], [(37 * i) % 130 for i in range(40)]),
    "bf16-64-8-rows": (16, 2, 64, 16, 2, BF16, [40, 24], [640, 96], [(53 * i) % 700 for i in range(64)]),
    "fp16-64-5-rows": (40, 8, 64, 16, 3, FP16, [17, 0, 30], [400, 32, 1600], [(29 * i) % 260 for i in range(47)]),
    "fp16-128-9-rows": (36, 4, 128, 16, 2, FP16, [33], [304], [(41 * i) % 400 for i in range(33)]),
    "bf16-128-16-rows": (64, 4, 128, 32, 2, BF16, [22, 10], [256, 64], [(77 * i) % 350 for i in range(32)]),
    "bf16-64-16-rows": (128, 8, 64, 8, 1, BF16, [14], [72], [(71 * i) % 500 for i in range(14)]),
    "fp16-64-12-rows-token-pages": (24, 2, 64, 1, 4, FP16, [45], [333], [(97 * i) % 600 for i in range(45)]),
    "one-head-each": (8, 8, 64, 16, 2, BF16, [20, 20], [160, 320], [(19 * i) % 200 for i in range(40)]),
    "groups-past-16": (32, 8, 64, 8, 3, FP16, [3, 2, 5] * 7, [8 * i for i in range(21)], [(7 * i) % 90 for i in range(70)]),
    "nothing-here-and-there": (32, 8, 128, 16, 2, BF16, [0, 8, 0, 17, 24, 0], [64, 0, 0, 48, 1040, 16], (EMPTY * 7)[:49]),
    "no-prefix-at-all": (32, 8, 128, 16, 2, BF16, [25, 25], [0, 0], (EMPTY * 7)[:50]),
    "a-thousand-requests": (8, 2, 64, 16, 2, BF16, [24, 1000], [640, 160], [(31 * i) % 70 for i in range(1024)]),
    "lengths-below-the-bound": (32, 8, 64, 16, 2, FP16, [40], [2048], [0] * 20 + [1] * 10 + [300] + [0] * 9),
}


@pytest.mark.parametrize("name", CASES)
def test_two_passes_match_64_bits(name):
    call = Call(CASES[name])
    out, lse = call()
    torch.cuda.synchronize()
    assert int(call.cache.d_status) == 0
    call.check(out, lse)
    for _ in range(3):  # the same bits every time
        again, lse2 = call()
        assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("name", ["bf16-128-4-rows", "fp16-64-12-rows-token-pages", "bf16-128-16-rows", "groups-past-16"])
def test_two_passes_in_a_graph(name):
    """Captured on another stream: replays follow the lengths and agree bit for bit with plain calls; two graphs side by side do not disturb each other."""
    call = Call(CASES[name], spare=40)
    call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for _ in range(2):
        out, lse = torch.empty_like(call.d_q), torch.empty(call.d_q.shape[:2], device="cuda")
        graph = torch.cuda.CUDAGraph()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            call(out=out, lse=lse)
        graphs.append(graph)
        outs.append((out, lse))
    other = torch.cuda.Stream()
    for turn in range(4):
        call.suffix = call.rng.integers(0, call.most + 1, len(call.suffix)).tolist() if turn else [0] * len(call.suffix)
        call.d_lens.copy_(torch.tensor(call.suffix, dtype=torch.int32))
        for out, lse in outs:
            out.fill_(7.0), lse.fill_(7.0)
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, (torch.cuda.current_stream(), other)):
            with torch.cuda.stream(stream):
                graph.replay()
                graph.replay()
        torch.cuda.synchronize()
        out, lse = call()
        for mine, my_lse in outs:
            assert torch.equal(mine, out) and torch.equal(my_lse, lse)
        call.check(out, lse, requests=6)
    assert int(call.cache.d_status) == 0


@pytest.mark.parametrize("offset", [0, 16, 48])
@pytest.mark.parametrize("name", ["bf16-128-4-rows", "fp16-64-5-rows", "bf16-64-16-rows"])
def test_two_passes_take_their_workspace_and_no_less(name, offset):
    call = Call(CASES[name])
    workspace, untouched = workspace_at(call.need, offset)
    out, lse = call(workspace=workspace)
    torch.cuda.synchronize()
    assert untouched()
    plain, plain_lse = call()
    assert torch.equal(out, plain) and torch.equal(lse, plain_lse) and int(call.cache.d_status) == 0
    with pytest.raises(cpkv.CpkvError) as e:
        call(workspace=workspace[:-16])
    assert e.value.code == cpkv.CPKV_ERR_CAPACITY


def test_two_passes_report_bad_pages_and_lengths():
    """A bad page of a prefix or of a suffix reads as zero rows, a length past the bound is clamped; each raises its bit."""
    name = "bf16-64-8-rows"
    for where, bad in [(where, bad) for where in ("prefix", "suffix") for bad in (-1, 0, 1 << 29)]:
        call = Call(CASES[name])
        ps, cp = call.case[3], call.case[4]
        if where == "prefix":
            lp, call.d_prefix[3] = int(call.prefix_pages[3]), bad
        else:
            lp, call.d_table[5, 1] = int(call.lists[5, 1]), bad
        assert call.suffix[5] > ps + 1
        out, lse = call()
        torch.cuda.synchronize()
        assert int(call.cache.d_status) == cpkv.STATUS_PAGE_OOB
        zeroed = qmodel.Pools(1, ps, cp, call.pools.row, BF16)
        zeroed.slabs = [s.copy() for s in call.pools.slabs]
        zeroed.slabs[lp % cp][lp // cp] = 0
        call.check(out, lse, requests=4, rows=zeroed)
    call = Call(CASES[name])
    call.d_lens[7], call.d_lens[9] = call.most + 1, -3
    call.suffix[7], call.suffix[9] = call.most, 0
    out, lse = call()
    assert int(call.cache.d_status) == cpkv.STATUS_OUT_CAPACITY
    call.check(out, lse, requests=64)


def test_two_passes_beside_other_work_of_the_stream():
    """The split pass starts early, but not before what stands on the stream ahead of the call: queries and rows that were just written."""
    call = Call(CASES["bf16-128-4-rows"])
    want, want_lse = call()
    torch.cuda.synchronize()
    rows = [t.clone() for t in call.cache.table.pools]
    lens, q = call.d_lens.clone(), call.d_q.clone()
    busy = torch.ones(4096, 4096, device="cuda")
    for _ in range(10):
        for t in call.cache.table.pools:
            t.zero_()
        call.d_lens.zero_(), call.d_q.zero_()
        busy = busy @ busy * 2.0**-12
        for t, r in zip(call.cache.table.pools, rows):
            t.copy_(r)
        call.d_lens.copy_(lens), call.d_q.copy_(q)
        out, lse = call()
        for t in call.cache.table.pools:  # and what follows waits for the call
            t.zero_()
        call.d_q.zero_()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        for t, r in zip(call.cache.table.pools, rows):
            t.copy_(r)
        call.d_q.copy_(q)


def test_two_passes_write_over_their_queries():
    call = Call(CASES["fp16-64-5-rows"])
    want, want_lse = call()
    q = call.d_q.clone()
    out, lse = call(q=q, out=q)
    assert out.data_ptr() == q.data_ptr() and torch.equal(out, want) and torch.equal(lse, want_lse)


def test_two_passes_keep_tiny_values():
    """Values of 2^-116 to 2^-110 in prefix and suffixes: the tile pass's parts and the split pass's meet in the join."""
    hq, hkv, d, ps, n = 32, 8, 64, 16, 40
    rng = np.random.default_rng(8)
    call = Call((hq, hkv, d, ps, 2, BF16, [n], [160], [(37 * i) % 130 for i in range(n)]))
    v = rng.standard_normal((d,))
    v[3] = 1.75
    v = np.clip(v, -1.75, 1.75)
    scale = 2.0 ** rng.integers(-124, -117, call.pools.slabs[0].shape[:2] + (hkv,))
    bytes_, one = qmodel.quantise(v[None])
    assert one[0] == 2.0**-8  # values below 2 in steps of 2^-8 e4m3 numbers: as large as scale * 2^8
    row = call.pools.row
    for slab in call.pools.slabs:
        slab[..., row.value_offset:row.value_offset + hkv * d] = np.tile(bytes_[0], hkv)
        slab[..., row.value_scale_offset:row.value_scale_offset + 4 * hkv] = scale.astype(np.float32).view(np.uint8).reshape(*slab.shape[:2], -1)
    call.cache = cache_of(call.pools, BF16)
    out, lse = call()
    want = model.shared(call.q, [n], [160], call.prefix_pages, call.lists, call.suffix, qmodel.Dense(call.pools), kv_heads=hkv, dim=d, scale=d**-0.5)
    check_scaled(out, lse, want, 110)
