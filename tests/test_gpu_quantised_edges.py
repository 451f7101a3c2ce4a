"""Quantised rows on the GPU: calls that are refused, empty caches, the ends of the number range."""
import bisect
from fractions import Fraction

import numpy as np
import pytest
import torch

import quantised_model as qmodel
import serving_model as model
from paged_kv_cache_compose_gb300 import cpkv
from paged_kv_cache_compose_gb300.cpkv import QuantisedRow
from test_gpu_quantised import cache_of, tensor, turns
from test_gpu_quantised_attend import KIND_NAMES, KINDS, want_window, window_case
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


# --------------------------------------------------------------------------- append: exact roundings

NUMBERS = [Fraction(float(x)) for x in qmodel.VALUES[:127]]
LIMIT = 448 * Fraction(2)**127  # what the largest scale reaches


def exact_bytes(x):
    """A group of rational numbers (None: infinite or no number) as (bytes, scale)."""
    x = [None if v is None or abs(v) > LIMIT else v for v in x]
    top = max([abs(v) for v in x if v is not None], default=Fraction(0))
    k = -126
    while 448 * Fraction(2)**k < top:
        k += 1
    out = []
    for v in x:
        if v is None:
            out.append(qmodel.NAN)
            continue
        z = abs(v) / Fraction(2)**k
        up = min(max(bisect.bisect_left(NUMBERS, z), 1), 126)
        low, high = z - NUMBERS[up - 1], NUMBERS[up] - z
        out.append((up - 1 if low < high or (low == high and up % 2 == 1) else up) | (128 if v < 0 else 0))
    return out, 2.0**k


def pair_of(case, rng, dtype):
    """One pair of a key's elements, and its cosine and sine (float32)."""
    eps = float(torch.finfo(dtype).eps)
    number = lambda: float(rng.choice([-1, 1])) * (1 + eps * int(rng.integers(1 / eps)))  # of the type, from 1 to 2
    angle = rng.uniform(-3.2, 3.2)
    c, s = np.float32(np.cos(angle)), np.float32(np.sin(angle))
    if case == "huge":  # the exact rotation passes 32 bits' range
        return number() * 2.0**127, number() * 2.0**127, c, s
    if case == "past":  # some of them past what any scale reaches
        return number() * 2.0**126, number() * 2.0**126, np.float32(c * 600), np.float32(s * 600)
    if case == "tiny":  # products' rests lie below 32 bits' range
        return number() * 2.0 ** int(rng.integers(-133, -117)), number() * 2.0 ** int(rng.integers(-133, -117)), c, s
    if case == "least":  # as small as the type's and the table's numbers get
        return number() * 2.0**-126, number() * 2.0**-126, np.float32(c * 2.0**-8), np.float32(s * 2.0**-8)
    if case == "ties":  # an odd multiple of half a step, but for a rest of 2^-47 and less of it that two products' rests leave
        tie = float(rng.choice([17, 19, 21, 23, 25, 27, 29, 31])) / 16 * 2.0 ** int(rng.integers(0, 7))
        a, b = abs(number()), abs(number())
        c = np.float32(tie / a)
        rest = Fraction(a) * Fraction(float(c)) - Fraction(tie)
        return a, b, c, np.float32(float(rest / Fraction(b)))
    # "cancels": both products are nearly the same
    a, b = number(), number()
    return a, b, c, np.float32(a * float(c) / b)


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "pairs"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("case, dtype", [("huge", BF16), ("past", BF16), ("tiny", BF16), ("least", BF16), ("ties", BF16), ("ties", FP16), ("cancels", BF16),
                                         ("cancels", FP16)], ids=lambda x: str(x).replace("torch.", ""))
def test_append_rounds_from_the_exact_value(case, dtype, d, interleaved):
    """Every byte and scale against rational arithmetic, where 32 bits are not enough."""
    n, hkv, ps, half = 24, 2, 16, d // 2
    rng = np.random.default_rng(d + interleaved)
    k, table = np.zeros((n, hkv, d)), np.zeros((n, d), np.float32)
    for t in range(n):
        for i in range(half):
            for h in range(hkv):  # heads share the angles: the last head's, whose pairs are as meant; the other's are turned by them
                a, b, c, s = pair_of(case, rng, dtype)
                one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
                k[t, h, one], k[t, h, two], table[t, i], table[t, half + i] = a, b, c, s
        if case in ("ties", "cancels"):  # a group of ordinary size: its largest element is 448, not turned
            k[t, :, [0, 1 if interleaved else half]] = np.array([[448.0], [0.0]])
            table[t, 0], table[t, half] = 1.0, 0.0
    keys = tensor(k, dtype)
    k = keys.double().numpy()  # (subnormal numbers have fewer bits)
    row = QuantisedRow.of(hkv, d)
    pools = qmodel.Pools(2, ps, 1, row, dtype)
    cache = cache_of(pools, dtype)
    cache.append_rotary(keys.cuda(), keys.cuda(), torch.arange(ps, ps + n).cuda(), torch.arange(n, dtype=torch.int32).cuda(), torch.from_numpy(table).cuda(),
                        interleaved=interleaved)
    torch.cuda.synchronize()
    assert int(cache.d_status) == 0
    got = cache.table.pools[0].cpu().numpy().reshape(-1, row.row_bytes)[ps:ps + n]
    bad = []
    for t in range(n):
        for h in range(hkv):
            y = [None] * d
            for i in range(half):
                one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
                a, b, c, s = (Fraction(float(v)) for v in (k[t, h, one], k[t, h, two], table[t, i], table[t, half + i]))
                y[one], y[two] = a * c - b * s, b * c + a * s
            want, scale = exact_bytes(y)
            at = row.key_offset + h * d
            mine, at_scale = got[t, at:at + d], row.key_scale_offset + 4 * h
            mine, want = np.where(mine == 128, 0, mine), np.where(np.array(want) == 128, 0, want)  # a zero has no sign
            if (mine != want).any() or float(np.ascontiguousarray(got[t, at_scale:at_scale + 4]).view(np.float32)[0]) != scale:
                bad.append((t, h, int((mine != want).sum())))
    assert not bad, f"{len(bad)} of {n * hkv} heads differ, first (token, head, bytes) {bad[0]}"
    if case == "past":
        assert (got[:, :2 * d] & 127 == qmodel.NAN).any()


# --------------------------------------------------------------------------- attention: many requests, many heads

def test_a_token_of_very_many_heads():
    """Rows read back without lengths of queries: one token a request, 1100 heads of it on one key head."""
    hq, d, ps = 1100, 64, 16
    case = (hq, 1, d, ps, 2, BF16, 70, 5, [1, 1], [300, 41])
    rng, pools, lists, q = window_case(case)
    args = (2, hq, 1, d, None, 300)
    assert cpkv.cpkv_attend_window_quantised_workspace_bytes(*args, window=70, sinks=5) > cpkv.cpkv_attend_window_workspace_bytes(*args, window=70, sinks=5)
    cache = cache_of(pools, BF16)
    out, lse = run_window(cache, case, q, lists)
    assert int(cache.d_status) == 0
    some = [0, 1, 255, 256, 700, 1023, 1024, 1099]
    want = want_window((len(some),) + case[1:], pools, lists, q[:, some])
    model.check(out[:, some], lse[:, some], want, BF16)


@pytest.mark.parametrize("tokens, window, dtype", [(20, 0, BF16), (20, 33, FP16), (60, 0, FP16), (60, 40, BF16)], ids=["tile", "tile-window", "unpacked", "unpacked-window"])
def test_more_requests_than_the_small_tables_hold(tokens, window, dtype):
    """Forty requests of different lengths, some without queries or keys, converted on the way or read back first."""
    hq, hkv, d, ps = 32, 2, 64, 8
    q_lens = [tokens - i % 3 if i % 13 else 0 for i in range(40)]
    kv_lens = [0 if i % 11 == 5 else n + (17 * i) % 90 for i, n in enumerate(q_lens)]
    case = (hq, hkv, d, ps, 3, dtype, window, 3 if window else 0, q_lens, kv_lens)
    rng, pools, lists, q = window_case(case)
    more = cpkv.cpkv_attend_window_quantised_workspace_bytes(40, hq, hkv, d, q_lens, max(kv_lens), window, case[7])
    assert (more > 40 * 60 * hkv * d * 4) == (tokens == 60)
    cache = cache_of(pools, dtype)
    out, lse = run_window(cache, case, q, lists)
    assert int(cache.d_status) == 0
    first = np.cumsum([0] + q_lens)
    for b in (1, 5, 12, 16, 17, 38):
        at = slice(first[b], first[b + 1])
        heads = [0, 15, 16, 31]  # of two key heads
        want = model.window(q[at][:, heads], [q_lens[b]], lists[b:b + 1], [kv_lens[b]], qmodel.Dense(pools),
                            kv_heads=2, dim=d, window=window, sinks=case[7], scale=d**-0.5)
        model.check(out[at][:, heads], lse[at][:, heads], want, dtype, f"request {b}")

