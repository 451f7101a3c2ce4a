"""Serving calls where their arguments sit at the edges of what the contract allows, against plain 64-bit implementations."""
import numpy as np
import pytest
import torch

import serving_model as model
from paged_kv_cache_compose_gb300 import cpkv
from paged_kv_cache_compose_gb300.runtime import PagedCache
from test_gpu_serving import BF16, FP16, page_tables, queries

pytestmark = pytest.mark.gpu


def workspace_at(need, offset):
    """`need` bytes at `offset` past a 256-byte boundary, and a check that nothing around them was written."""
    whole = torch.full((offset + need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    assert whole.data_ptr() % 256 == 0

    def untouched():
        return bool((whole[:offset] == 0xA5).all()) and bool((whole[offset + need:] == 0xA5).all())

    return whole[offset:offset + need], untouched


@pytest.mark.parametrize("offset", [0, 16, 32, 48])
@pytest.mark.parametrize("q_lens, kv_lens", [([11], [4000]), ([1, 1], [3000, 900])], ids=["tile", "split"])
def test_window_workspace_at_any_multiple_of_16(q_lens, kv_lens, offset):
    """The workspace that the sizing call asks for, wherever it begins, is enough and all that is written."""
    hq, hkv, d, ps = 12, 1, 128, 64
    rng = np.random.default_rng(offset)
    lists, n_pages = page_tables(rng, kv_lens, ps)
    pools = model.Pools(rng, n_pages, ps, 2, 2 * hkv * d, BF16)
    q = queries(rng, sum(q_lens), hq, d, BF16)
    cache = PagedCache(pools.cuda(), page_size=ps, kv_heads=hkv, key_dim=d)
    need = cpkv.cpkv_attend_window_workspace_bytes(len(q_lens), hq, hkv, d, q_lens, max(kv_lens))
    assert need > 0
    workspace, untouched = workspace_at(need, offset)
    d_q = q.cuda()
    out, lse = torch.empty_like(d_q), torch.empty(q.shape[:2], device="cuda")
    cpkv.cpkv_attend_window(d_q, q_lens, torch.from_numpy(lists).cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda(),
                            table=cache.table, kv_heads=hkv, max_kv_len=max(kv_lens), window=0, sinks=0, scale=d**-0.5, out=out,
                            lse=lse, workspace=workspace, d_status=cache.d_status)
    torch.cuda.synchronize()
    assert int(cache.d_status) == 0 and untouched()
    model.check(out, lse, model.window(q, q_lens, lists, kv_lens, pools, kv_heads=hkv, dim=d, window=0, sinks=0, scale=d**-0.5), BF16)


@pytest.mark.parametrize("offset", [0, 16, 32, 48])
@pytest.mark.parametrize("requests", [24, 2], ids=["tile", "split"])
def test_shared_workspace_at_any_multiple_of_16(requests, offset):
    hq, hkv, d, ps = 8, 2, 64, 16
    sizes, prefix, suffix = [requests], [800], [1 + 7 * i for i in range(requests)]
    rng = np.random.default_rng(offset)
    lists, n_pages = page_tables(rng, prefix + suffix, ps)
    pools = model.Pools(rng, n_pages, ps, 2, 2 * hkv * d, FP16)
    prefix_pages = lists[0, :prefix[0] // ps].astype(np.int32)
    q = queries(rng, requests, hq, d, FP16)
    cache = PagedCache(pools.cuda(), page_size=ps, kv_heads=hkv, key_dim=d)
    need = cpkv.cpkv_attend_shared_workspace_bytes(requests, hq, hkv, d, sizes, prefix, max(suffix))
    workspace, untouched = workspace_at(need, offset)
    d_q = q.cuda()
    out, lse = torch.empty_like(d_q), torch.empty(q.shape[:2], device="cuda")
    cpkv.cpkv_attend_shared(d_q, sizes, prefix, torch.from_numpy(prefix_pages).cuda(), torch.from_numpy(lists[1:]).cuda(),
                            torch.tensor(suffix, dtype=torch.int32).cuda(), table=cache.table, kv_heads=hkv,
                            max_suffix_len=max(suffix), scale=d**-0.5, out=out, lse=lse, workspace=workspace, d_status=cache.d_status)
    torch.cuda.synchronize()
    assert int(cache.d_status) == 0 and untouched()
    want = model.shared(q, sizes, prefix, prefix_pages, lists[1:], suffix, pools, kv_heads=hkv, dim=d, scale=d**-0.5)
    model.check(out, lse, want, FP16)


def test_calls_run_with_the_pools_device_current():
    """Every call makes the pools' device current before it looks at anything else: of a device that is not there, the switch itself fails."""
    cache = PagedCache([torch.zeros(4, 16, 256, dtype=BF16, device="cuda")], page_size=16, kv_heads=2, key_dim=64)
    rows = torch.zeros(0, 2, 64, dtype=BF16, device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    turns, pages = torch.ones(8, 64, device="cuda"), torch.zeros(0, 1, dtype=torch.int32, device="cuda")

    def calls():
        cache.append_rotary(rows, rows, none.long(), none, turns)
        cache.attend_window(rows, None, pages, none, max_kv_len=16, out=rows)
        cache.attend_shared(rows, [], [], none, pages, none, max_suffix_len=16, out=rows)

    calls()
    missing = torch.cuda.device_count()
    cache.table._table.device = missing
    stream = torch.cuda.current_stream().cuda_stream
    for call in (lambda: cache.append_rotary(rows, rows, none.long(), none, turns, stream=stream),
                 lambda: cache.attend_window(rows, None, pages, none, max_kv_len=16, out=rows, stream=stream),
                 lambda: cache.attend_shared(rows, [], [], none, pages, none, max_suffix_len=16, out=rows, stream=stream)):
        with pytest.raises(RuntimeError) as e:
            call()
        assert not isinstance(e.value, cpkv.CpkvError)  # which is a tensor's refusal
    assert torch.cuda.current_device() == 0
    cache.table._table.device = 0
    calls()
    assert int(cache.d_status) == 0


def test_status_words_and_workspaces_that_calls_refuse():
    """A status word that is no int32 or is empty, and memory of the host: refused before anything is launched."""
    cache = PagedCache([torch.zeros(4, 16, 256, dtype=BF16, device="cuda")], page_size=16, kv_heads=2, key_dim=64)
    k = torch.zeros(1, 2, 64, dtype=BF16, device="cuda")
    one, turns, pages = torch.ones(1, dtype=torch.int32, device="cuda"), torch.ones(8, 64, device="cuda"), torch.ones(1, 1, dtype=torch.int32, device="cuda")
    out, room = torch.empty_like(k), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")

    def append(d_status, workspace):
        cpkv.cpkv_append_rotary(k, k, 16 * one.long(), one, turns, table=cache.table, d_status=d_status)

    def window(d_status, workspace):
        cpkv.cpkv_attend_window(k, None, pages, one, table=cache.table, kv_heads=2, max_kv_len=16, window=0, sinks=0, scale=0.1, out=out,
                                lse=None, workspace=workspace, d_status=d_status)

    def shared(d_status, workspace):
        cpkv.cpkv_attend_shared(k, [1], [0], one[:0], pages, one, table=cache.table, kv_heads=2, max_suffix_len=16, scale=0.1, out=out, lse=None,
                                workspace=workspace, d_status=d_status)

    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    for call in (append, window, shared):
        call(word, room)
        for bad in (word.to(torch.int8), word.float(), word.long(), word[:0], word.cpu(), None):
            with pytest.raises(cpkv.CpkvError):
                call(bad, room)
    for call in (window, shared):
        for bad in (room.cpu(), room[::2]):
            with pytest.raises(cpkv.CpkvError):
                call(word, bad)
    torch.cuda.synchronize()
    assert int(word) == 0


class Recorder:
    """The compiled calls of a handle, with the workspaces that they were given."""

    def __init__(self, native):
        self.native, self.spans = native, []

    def __getattr__(self, name):
        if name == "captures":
            return self.native.captures

        def call(*args):
            rc = getattr(self.native, name)(*args)
            if rc == 0 and args[12] is not None:
                self.spans.append((args[12].data_ptr(), args[12].data_ptr() + args[12].numel()))
            return rc

        return call


def decode_batch(seed=0):
    """A decode step whose rows are cut into parts: inputs on the GPU and the wanted result."""
    hq, hkv, d, ps, kv_lens = 8, 2, 128, 16, [3000, 1700, 2500]
    rng = np.random.default_rng(seed)
    lists, n_pages = page_tables(rng, kv_lens, ps)
    pools = model.Pools(rng, n_pages, ps, 2, 2 * hkv * d, BF16)
    cache = PagedCache(pools.cuda(), page_size=ps, kv_heads=hkv, key_dim=d)
    q = [queries(rng, 3, hq, d, BF16) for _ in range(3)]
    want = [model.window(x, [1] * 3, lists, kv_lens, pools, kv_heads=hkv, dim=d, window=0, sinks=0, scale=d**-0.5) for x in q]
    table, lens = torch.from_numpy(lists).cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda()

    def step(k_q, out, lse, **more):
        return cache.attend_window(k_q, None, table, lens, max_kv_len=3000, out=out, lse=lse, **more)

    d_q = [x.cuda() for x in q]
    outs = [(torch.zeros_like(x), torch.zeros(3, hq, device="cuda")) for x in d_q]
    return cache, step, d_q, outs, want


@pytest.mark.parametrize("explicit", [False, True])
def test_captured_calls_have_workspaces_of_their_own(explicit):
    """Two graphs captured on one stream, and an eager call there, take memory apart from each other."""
    cache, step, q, outs, want = decode_batch()
    cache._native = recorder = Recorder(cache._native)
    stream = torch.cuda.Stream()
    graphs, more = [torch.cuda.CUDAGraph() for _ in range(2)], dict(stream=stream) if explicit else {}
    with torch.cuda.stream(stream):
        step(q[2], *outs[2])
    for graph, x, out in zip(graphs, q, outs):
        with torch.cuda.graph(graph, stream=stream):
            step(x, *out, **more)
    with torch.cuda.stream(stream):
        step(q[2], *outs[2])
    torch.cuda.synchronize()
    eager, first, second, again = recorder.spans
    assert again == eager
    for a, b in ((eager, first), (eager, second), (first, second)):
        assert a[1] <= b[0] or b[1] <= a[0]
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        model.check(*out, w, BF16)
    assert int(cache.d_status) == 0


def test_replays_and_eager_calls_side_by_side():
    cache, step, q, outs, want = decode_batch(1)
    capture, one, two = (torch.cuda.Stream() for _ in range(3))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph, x, out in zip(graphs, q, outs):
        with torch.cuda.graph(graph, stream=capture):
            for _ in range(20):
                step(x, *out)
    torch.cuda.synchronize()
    for _ in range(30):
        for side, graph in ((one, graphs[0]), (two, graphs[1])):
            with torch.cuda.stream(side):
                graph.replay()
        with torch.cuda.stream(capture):
            for _ in range(10):
                step(q[2], *outs[2])
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        model.check(*out, w, BF16)


def test_a_workspace_of_the_caller():
    """The caller's memory is used as it is, and refused when it is too small."""
    cache, step, q, outs, want = decode_batch(2)
    need = cpkv.cpkv_attend_window_workspace_bytes(3, 8, 2, 128, None, 3000)
    cache._native = recorder = Recorder(cache._native)
    mine = torch.empty(need, dtype=torch.uint8, device="cuda")
    step(q[0], *outs[0], workspace=mine)
    assert recorder.spans == [(mine.data_ptr(), mine.data_ptr() + need)]
    model.check(*outs[0], want[0], BF16)
    with pytest.raises(cpkv.CpkvError):
        step(q[0], *outs[0], workspace=mine[:-1])
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step(q[1], *outs[1], workspace=mine)
    graph.replay()
    torch.cuda.synchronize()
    assert recorder.spans[1] == recorder.spans[0]
    model.check(*outs[1], want[1], BF16)


@pytest.mark.parametrize("d, tokens", [(64, 64), (128, 64), (64, 256), (128, 2048), (64, 60000)])
def test_blocks_that_give_up_leave_the_gpu_usable(d, tokens):
    """Waits that run out at the start and in the middle of long items: the status says so, and what runs next is right."""
    pages = 1024
    rows = torch.zeros(pages, 64, 2 * d, dtype=BF16, device="cuda")
    table, lens = torch.arange(pages, dtype=torch.int32, device="cuda"), torch.tensor([64 * pages], dtype=torch.int32, device="cuda")
    q = torch.zeros(tokens, d, dtype=BF16, device="cuda")
    out = torch.empty_like(q)
    for wait_ns in (0, 1000, 10_000, 50_000, 10**9):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        cpkv.cpkv_selftest_attend_timeout(rows, table, lens, q, out, wait_ns, status)
        torch.cuda.synchronize()
        # 65536 keys take hundreds of us: no block gets through without a wait of 50; none of them waits for a second
        assert int(status) == (0 if wait_ns == 10**9 else cpkv.STATUS_TIMEOUT), wait_ns
        assert wait_ns < 10**9 or bool((out == 0).all())
        cache, step, d_q, outs, want = decode_batch(3)
        step(d_q[0], *outs[0])
        long = cache.attend_window(d_q[1].expand(3, -1, -1).contiguous(), [3], torch.arange(1, 180, dtype=torch.int32, device="cuda")[None],
                                   torch.tensor([2500], dtype=torch.int32, device="cuda"), max_kv_len=2500)
        torch.cuda.synchronize()
        model.check(*outs[0], want[0], BF16)
        assert bool(long.isfinite().all()) and int(cache.d_status) == 0


def test_infinite_values_beside_very_many_keys():
    """One NaN and one infinity among 300 000 keys, near the end: the rows that do not see them are worked out again in
    time, whole items long, and stay right."""
    hq, hkv, d, ps, kv, nq = 32, 8, 128, 64, 300_000, 2560  # 320 items, each over all keys
    gen = torch.Generator(device="cuda").manual_seed(1)
    pages = -(-kv // ps)
    pool = torch.randn(pages, ps, 2 * hkv * d, dtype=BF16, device="cuda", generator=gen)
    table = torch.randperm(pages, device="cuda", generator=gen).int()[None]
    q = torch.randn(nq, hq, d, dtype=BF16, device="cuda", generator=gen)

    def spoil(key, head, element, value):
        pool[int(table[0, key // ps]), key % ps, (hkv + head) * d + element] = value

    # (key, head, element): the last token sees the first; tokens from kv - 1000 on see the second
    spoil(kv - 1, 2, 5, float("nan"))
    spoil(kv - 1000, 6, 77, float("inf"))
    cache = PagedCache([pool], page_size=ps, kv_heads=hkv, key_dim=d, dense=True)
    lse = torch.empty(nq, hq, device="cuda")
    out = cache.attend_window(q, [nq], table, torch.tensor([kv], dtype=torch.int32, device="cuda"), max_kv_len=kv, lse=lse)
    torch.cuda.synchronize()
    assert int(cache.d_status) == 0
    want = torch.ones_like(out, dtype=torch.bool)
    want[nq - 1, 8:12, 5] = False
    want[nq - 1000:, 24:28, 77] = False
    assert torch.equal(out.isfinite(), want) and bool(lse.isfinite().all())
    rows = pool[table[0].long()].view(-1, 2, hkv, d)[:kv]
    for token, head in [(nq - 2, 9), (nq - 64, 11), (nq - 30, 8), (nq - 1001, 25), (nq - 1024, 24), (nq - 1001, 9), (nq - 1, 0)]:
        seen, c = kv - nq + token + 1, head // 4
        k, v = rows[:seen, 0, c].double(), rows[:seen, 1, c].double()
        s = k @ q[token, head].double() * d**-0.5
        e = torch.logsumexp(s, 0)
        w = torch.exp(s - e)
        model.check(out[token, head], lse[token, head], ((w @ v).cpu(), e.cpu(), (w @ v.abs()).cpu()), BF16)


@pytest.mark.parametrize("q_lens, kv_lens", [([1, 1, 1], [3, 700, 0]), ([5, 5], [2, 0]), ([40, 3], [20, 300]), ([64], [1])],
                         ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 6, "longest"])
def test_windows_beyond_every_key_are_none(q_lens, kv_lens, window):
    """Requests shorter than their queries under windows near 2^31: positions below 0 less the window."""
    hq, hkv, d, ps = 8, 2, 64, 16
    rng = np.random.default_rng(sum(kv_lens))
    lists, n_pages = page_tables(rng, kv_lens, ps)
    pools = model.Pools(rng, n_pages, ps, 2, 2 * hkv * d, BF16)
    q = queries(rng, sum(q_lens), hq, d, BF16)
    cache = PagedCache(pools.cuda(), page_size=ps, kv_heads=hkv, key_dim=d)
    table, lens = torch.from_numpy(lists).cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda()
    results = []
    for w, sinks in ((0, 0), (max(kv_lens) if window == "longest" else window, 0), (max(kv_lens) if window == "longest" else window, 2**31 - 1)):
        lse = torch.full((sum(q_lens), hq), 7.0, device="cuda")
        out = cache.attend_window(q.cuda(), q_lens, table, lens, max_kv_len=max(kv_lens), window=w, sinks=sinks, lse=lse)
        torch.cuda.synchronize()
        model.check(out, lse, model.window(q, q_lens, lists, kv_lens, pools, kv_heads=hkv, dim=d, window=0, sinks=0, scale=d**-0.5), BF16)
        results.append((out, lse))
    for out, lse in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(lse, results[0][1])
    assert int(cache.d_status) == 0


@pytest.mark.parametrize("nq, hq", [(1, 8), (3, 8), (11, 24)], ids=["split", "split-queries", "tile"])
def test_an_infinite_value_of_tiny_weight_in_another_part(nq, hq):
    """The first key's score leaves nothing to the others in 32 bits; an infinity among them still reaches the rows that see it."""
    hkv, d, ps, kv = 2, 128, 16, 3000
    rng = np.random.default_rng(nq)
    lists, n_pages = page_tables(rng, [kv], ps)
    pools = model.Pools(rng, n_pages, ps, 2, 2 * hkv * d, BF16)
    q = queries(rng, nq, hq, d, BF16)
    q[..., 0] = 64.0
    first = pools.row(int(lists[0, 0]), 0)
    first[0] = first[d] = 64.0  # a score of 64 * 64 / sqrt(128) more than the others'
    key = 2000
    pools.row(int(lists[0, key // ps]), key % ps)[hkv * d + d + 7] = float("inf")
    cache = PagedCache(pools.cuda(), page_size=ps, kv_heads=hkv, key_dim=d)
    out = cache.attend_window(q.cuda(), [nq], torch.from_numpy(lists).cuda(), torch.tensor([kv], dtype=torch.int32).cuda(), max_kv_len=kv)
    want = torch.ones(nq, hq, d, dtype=torch.bool)
    want[:, hq // 2:, 7] = False
    assert torch.equal(out.cpu().isfinite(), want)


@pytest.mark.parametrize("requests", [2, 24], ids=["split", "tile"])
def test_an_infinite_value_of_tiny_weight_in_a_suffix(requests):
    hq, hkv, d, ps, prefix = 8, 1, 64, 16, 480
    suffix = [1 + 3 * i for i in range(requests)]
    rng = np.random.default_rng(requests)
    lists, n_pages = page_tables(rng, [prefix] + suffix, ps)
    pools = model.Pools(rng, n_pages, ps, 2, 2 * hkv * d, FP16)
    q = queries(rng, requests, hq, d, FP16)
    q[..., 0] = 64.0
    pools.row(int(lists[0, 0]), 0)[0] = 64.0
    pools.row(int(lists[2, 0]), 1)[hkv * d + 3] = -float("inf")  # the second request's
    cache = PagedCache(pools.cuda(), page_size=ps, kv_heads=hkv, key_dim=d)
    out = cache.attend_shared(q.cuda(), [requests], [prefix], torch.from_numpy(lists[0, :prefix // ps].astype(np.int32)).cuda(),
                              torch.from_numpy(lists[1:]).cuda(), torch.tensor(suffix, dtype=torch.int32).cuda(), max_suffix_len=max(suffix))
    want = torch.ones(requests, hq, d, dtype=torch.bool)
    want[1, :, 3] = False
    assert torch.equal(out.cpu().isfinite(), want)


@pytest.mark.parametrize("dtype", [FP16, BF16])
@pytest.mark.parametrize("nq, hq, kv", [(1, 2, 3000), (3, 2, 3000), (64, 1, 3000), (300, 1, 900), (1, 2, 200)],
                         ids=["split", "split-queries", "parts", "tile", "few-keys"])
def test_many_small_weights_beside_one_large(nq, hq, kv, dtype):
    """One key's weight is 2^25 times the others', whose values are all that the result is made of."""
    d, ps = 64, 16
    rng = np.random.default_rng(kv)
    lists, n_pages = page_tables(rng, [kv], ps)
    pools = model.Pools(rng, n_pages, ps, 2, 2 * d, dtype)
    for s in pools.slabs:
        s[..., :d] = 0.0
        s[..., d:] = 1.0
    first = pools.row(int(lists[0, 0]), 0)
    first[0], first[d:] = 8.75, 0.0
    q = torch.zeros(nq, hq, d, dtype=dtype)
    q[..., 0] = 16.0
    want = model.window(q, [nq], lists, [kv], pools, kv_heads=1, dim=d, window=0, sinks=0, scale=d**-0.5)
    cache = PagedCache(pools.cuda(), page_size=ps, kv_heads=1, key_dim=d)
    lse = torch.empty(nq, hq, device="cuda")
    out = cache.attend_window(q.cuda(), [nq], torch.from_numpy(lists).cuda(), torch.tensor([kv], dtype=torch.int32).cuda(), max_kv_len=kv, lse=lse)
    model.check(out, lse, want, dtype)


def small_calls():
    cache = PagedCache([torch.zeros(4, 16, 256, dtype=BF16, device="cuda")], page_size=16, kv_heads=2, key_dim=64)
    k = torch.zeros(1, 2, 64, dtype=BF16, device="cuda")
    one, turns = torch.ones(1, dtype=torch.int32, device="cuda"), torch.ones(8, 64, device="cuda")
    pages = torch.ones(1, 1, dtype=torch.int32, device="cuda")
    return cache, dict(
        append=lambda x=k, **more: cache.append_rotary(x, x, 16 * one.long(), one, turns, **more),
        window=lambda x=k, lens=None, **more: cache.attend_window(x, lens, pages, one, max_kv_len=16, **more),
        shared=lambda x=k, lens=(1,), **more: cache.attend_shared(x, lens, [0], one[:0], pages, one, max_suffix_len=16, **more))


def test_streams_and_numbers_that_are_none():
    """A stream that is no handle, a scale that is no number: an exception before anything is launched."""
    cache, calls = small_calls()
    for name, call in calls.items():
        for stream in (-1, 1 << 70):
            with pytest.raises(Exception):
                call(stream=stream)
    for name in ("window", "shared"):
        with pytest.raises(TypeError):
            calls[name](scale="1")
    torch.cuda.synchronize()
    assert int(cache.d_status) == 0


def test_lengths_that_are_refused_let_their_array_go():
    """An array of lengths of another type is free again after the exception."""
    _, calls = small_calls()
    for name in ("window", "shared"):
        for bad in (np.ones(1, np.float64), np.array([1.5], np.float32)):
            with pytest.raises(TypeError):
                calls[name](lens=bad)
            bad.resize(3, refcheck=False)  # raises while a buffer of it is held
        held = bytearray(b"\x01")
        calls[name](lens=held)
        held.append(1)  # likewise


def test_a_single_token_has_no_stride():
    """A token taken out of a tensor whose rows are no multiple of 16 bytes apart."""
    _, calls = small_calls()
    rows = torch.zeros(1, 132, dtype=BF16, device="cuda")  # one row of 132 elements, of which the first 128 are the heads
    odd = rows.as_strided((1, 2, 64), (132, 64, 1))
    assert odd.stride(0) == 132
    for call in calls.values():
        call(odd)


@pytest.mark.parametrize("q_lens, heads", [([1, 1], 4), ([1] * 60, 4), ([2, 0, 3], 4), ([40, 300], 4)], ids=["few-keys", "line", "queries", "tile"])
def test_requests_without_any_keys(q_lens, heads):
    """No request has a key, nor the table a page: zeros and -infinity."""
    hkv, d = 4, 64
    cache = PagedCache([torch.ones(4, 16, 2 * hkv * d, dtype=BF16, device="cuda")], page_size=16, kv_heads=hkv, key_dim=d)
    q = torch.ones(sum(q_lens), heads, d, dtype=BF16, device="cuda")
    lse = torch.zeros(q.shape[:2], device="cuda")
    for pages, most in ((0, 0), (1, 16)):
        out = cache.attend_window(q, q_lens, torch.full((len(q_lens), pages), -7, dtype=torch.int32, device="cuda"),
                                  torch.zeros(len(q_lens), dtype=torch.int32, device="cuda"), max_kv_len=most, lse=lse.zero_(), window=3, sinks=2)
        torch.cuda.synchronize()
        assert int(cache.d_status) == 0 and bool((out == 0).all()) and bool(torch.isneginf(lse).all())
