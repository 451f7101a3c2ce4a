"""Quantised rows on the GPU against plain 64-bit implementations: written, read back."""
import numpy as np
import pytest
import torch

import quantised_model as model
from paged_kv_cache_compose_gb300 import cpkv
from paged_kv_cache_compose_gb300.cpkv import QuantisedRow
from paged_kv_cache_compose_gb300.runtime import QuantisedCache

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16


def turns(rng, positions, rot):
    angle = rng.uniform(-3, 3, (positions, rot // 2))
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def tensor(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x).astype(np.float32)).to(dtype)


def cache_of(pools, dtype, **more):
    row = pools.row
    return QuantisedCache(pools.cuda(), page_size=pools.ps, kv_heads=row.kv_heads, key_dim=row.key_dim, value_dim=row.value_dim, dtype=dtype,
                          keep_keys=bool(row.keep_keys), row=row, **more)


def same_rows(got, want, pools):
    """Slabs byte for byte, but that a zero has no sign."""
    for a, b in zip(got, want):
        a = a.cpu().numpy()
        for raw in (a, b):
            assert raw.shape == b.shape
        row = pools.row
        a, b = a.reshape(-1, a.shape[-1]).copy(), b.reshape(-1, b.shape[-1]).copy()
        for at, n in [(row.value_offset, row.kv_heads * row.value_dim)] + [(row.key_offset, row.kv_heads * row.key_dim)] * (not row.keep_keys):
            for raw in (a, b):
                part = raw[:, at:at + n]
                part[part == 128] = 0
        if row.keep_keys:  # both rounded once, one of them from 32 bits: products and sum are off by 3 * 2^-24 of a pair's length, 2^-21 of the head's largest
            ka, kb = pools.rows(a)[0], pools.rows(b)[0]
            u = torch.finfo(pools.dtype).eps / 2
            assert (np.abs(ka - kb) <= 2 * u * np.abs(kb) + 2.0**-21 * np.abs(kb).max(-1, keepdims=True)).all()
            a[:, row.key_offset:row.key_offset + 2 * row.kv_heads * row.key_dim] = 0
            b[:, row.key_offset:row.key_offset + 2 * row.kv_heads * row.key_dim] = 0
        bad = np.argwhere(a != b)
        assert not len(bad), f"{len(bad)} bytes differ, first row and byte {bad[0].tolist()}: {a[tuple(bad[0])]:#x}, not {b[tuple(bad[0])]:#x}"


APPEND = [  # n, q heads, kv heads, key dim, value dim, keep keys, rot, interleaved, axes, ps, cp, dtype
    (1, 8, 1, 64, 64, False, 64, False, 1, 16, 1, BF16),
    (37, 4, 2, 128, 128, False, 128, False, 1, 16, 2, BF16),
    (37, 4, 2, 128, 128, False, 96, True, 1, 1, 8, FP16),
    (130, 5, 1, 64, 64, False, 32, False, 3, 64, 3, FP16),
    (65, 8, 8, 64, 64, False, 48, True, 3, 16, 2, BF16),
    (33, 16, 1, 64, 512, True, 64, True, 1, 16, 2, BF16),
    (33, 0, 1, 72, 128, True, 16, False, 1, 5, 2, FP16),
    (9, 3, 3, 128, 256, False, 128, False, 4, 7, 1, FP16),
    (20, 2, 5, 128, 64, False, 0, False, 1, 16, 2, BF16),
    (11, 3, 3, 64, 64, False, 64, False, 1, 16, 2, BF16),
    (9000, 8, 2, 128, 128, False, 64, False, 1, 64, 8, BF16),   # two heads a thread
    (9001, 7, 3, 64, 64, False, 48, True, 3, 64, 8, FP16),
    (9001, 16, 1, 64, 512, True, 64, True, 1, 64, 8, BF16),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(map(str, c)))
def test_append_quantises_the_exact_rotation(case):
    n, hq, hkv, dk, dv, keep, rot, interleaved, axes, ps, cp, dtype = case
    rng = np.random.default_rng(n + rot)
    row = QuantisedRow.of(hkv, dk, dv, keep)
    n_pages = -(-n // ps) + 3
    pools = model.Pools(n_pages, ps, cp, row, dtype, row.row_bytes + 16)  # 16 bytes behind each row that are left alone
    for slab in pools.slabs:
        slab[:] = rng.integers(0, 256, slab.shape) & 0x77  # numbers in any of the types
    slots = ps + rng.permutation(n_pages * ps)[:n]
    slots[::7] = np.where(np.arange(n)[::7] % 2 == 0, slots[::7], -1)  # some padding tokens
    positions = rng.integers(0, 500, (axes, n)).astype(np.int32)
    axis = rng.integers(0, axes, rot // 2).tolist()
    table = turns(rng, 500, rot) if rot else np.zeros((500, 0), np.float32)
    table[0] = np.concatenate([np.ones(rot // 2), np.zeros(rot // 2)])  # position 0 turns nothing: ties between two numbers
    positions[:, ::3] = 0
    size = np.exp(3 * rng.standard_normal((n, 1, 1)))
    k, v, q = (tensor(rng.standard_normal((n, h, d)) * s, dtype) for h, d, s in ((hkv, dk, size), (hkv, dv, size), (max(hq, 1), dk, 1.5)))
    cache = cache_of(pools, dtype)
    pos = torch.from_numpy(positions).cuda()
    got_q = cache.append_rotary(k.cuda(), v.cuda(), torch.from_numpy(slots).cuda(), pos if axes > 1 else pos[0], torch.from_numpy(table).cuda(),
                                q=q.cuda() if hq else None, axis_of_freq=axis if axes > 1 else None, interleaved=interleaved)
    torch.cuda.synchronize()
    assert int(cache.d_status) == 0
    turned = model.rotated(k.double().numpy(), table, positions, axis, interleaved)
    for t, slot in enumerate(slots):
        if slot >= 0:
            pools.put(slot // ps, slot % ps, turned[t], v[t].double().numpy())
    same_rows(cache.table.pools, pools.slabs, pools)
    if hq:
        want = model.rotated(q.double().numpy(), table, positions, axis, interleaved)
        # one rounding of a sum of two 32-bit products of values below 16: half a step, and 2^-19 for the products
        assert (np.abs(got_q.double().cpu().numpy() - want) <= model.torch.finfo(dtype).eps / 2 * np.abs(want) + 2.0**-19).all()


def test_append_of_what_e4m3_cannot_hold():
    """Zeros, subnormal and huge groups, infinities and NaNs: those become no number, the others keep their scale."""
    ps, d, n = 16, 128, 12
    row = QuantisedRow.of(1, d)
    rng = np.random.default_rng(3)
    x = rng.standard_normal((n, 1, d))
    x[0] = 0
    x[1] *= 2.0**-133
    x[2] *= 2.0**120
    x[3, 0, 5], x[3, 0, 6], x[3, 0, 77] = np.inf, -np.inf, np.nan
    x[4] = np.inf
    x[5] = 448.0
    x[6] = np.linspace(-449, 449, d)
    x[7] = 2.0**-9 * np.arange(d) / 16  # around the smallest numbers beside a large one
    x[7, 0, 0] = 448
    x[8] = -0.0
    k, v = tensor(x, BF16), tensor(x[::-1], BF16)
    pools = model.Pools(3, ps, 1, row, BF16)
    cache = cache_of(pools, BF16)
    slots = torch.arange(ps, ps + n)
    cache.append_rotary(k.cuda(), v.cuda(), slots.cuda(), torch.zeros(n, dtype=torch.int32, device="cuda"), torch.zeros(1, 0, device="cuda"))
    for t in range(n):
        pools.put(1, t, k[t].double().numpy(), v[t].double().numpy())
    same_rows(cache.table.pools, pools.slabs, pools)
    # rotated by nothing: the same (an infinity turns its pair into no numbers)
    again = cache_of(model.Pools(3, ps, 1, row, BF16), BF16)
    one = torch.cat([torch.ones(1, 64), torch.zeros(1, 64)], 1).cuda()
    finite = [t for t in range(n) if t not in (3, 4, 7, 8)]
    again.append_rotary(k[finite].cuda(), v[finite].cuda(), slots[finite].cuda(), torch.zeros(len(finite), dtype=torch.int32, device="cuda"), one)
    want = [torch.from_numpy(s) for s in pools.slabs]
    assert all(torch.equal(again.table.pools[0][1, t].cpu() & 0x7F, want[0][1, t] & 0x7F) for t in finite)


def test_append_reports_bad_slots_and_positions():
    rng = np.random.default_rng(6)
    ps, d = 4, 64
    row = QuantisedRow.of(1, d)
    table = torch.ones(10, d, device="cuda")
    k, v, q = (tensor(rng.standard_normal((4, 1, d)), BF16).cuda() for _ in range(3))
    for slots, pos, bit in [([4, 2, 8, 12], [0, 1, 2, 3], cpkv.STATUS_PAGE_OOB), ([4, 24, 8, 12], [0, 1, 2, 3], cpkv.STATUS_PAGE_OOB),
                            ([4, 1 << 40, 8, 12], [0, 1, 2, 3], cpkv.STATUS_PAGE_OOB),
                            ([4, 20, 8, 12], [0, 10, 2, 3], cpkv.STATUS_POS_OOB), ([4, 20, 8, 12], [0, -1, 2, 3], cpkv.STATUS_POS_OOB)]:
        pools = model.Pools(5, ps, 2, row, BF16)
        cache = cache_of(pools, BF16)
        got = cache.append_rotary(k, v, torch.tensor(slots).cuda(), torch.tensor(pos, dtype=torch.int32).cuda(), table, q=q)
        assert int(cache.d_status) == bit
        assert bool((got[1] == 0).all()) == (bit == cpkv.STATUS_POS_OOB)
        for page in range(1, 6):
            rows = cache.table.pools[page % 2][page // 2]
            assert not bool(rows[1:].any()) and bool(rows[0].any()) == (page in (1, 2, 3))


READ = [  # n, kv heads, key dim, value dim, keep keys, ps, cp, dtype
    (1, 1, 64, 64, False, 16, 1, BF16), (77, 2, 128, 128, False, 1, 8, FP16), (300, 3, 64, 64, False, 5, 2, BF16), (41, 1, 64, 512, True, 64, 2, BF16),
    (19, 1, 72, 128, True, 16, 3, FP16), (50, 2, 128, 256, False, 16, 2, BF16), (9001, 8, 128, 128, False, 64, 8, BF16), (20001, 1, 64, 512, True, 64, 2, BF16),
]


@pytest.mark.parametrize("case", READ, ids=lambda c: "-".join(map(str, c)))
def test_read_rows(case):
    """Rows in any order, named twice, negative (zeros), into slices of one buffer; scales of any size."""
    n, hkv, dk, dv, keep, ps, cp, dtype = case
    rng = np.random.default_rng(n)
    row = QuantisedRow.of(hkv, dk, dv, keep)
    n_pages = min(-(-n // ps), 40) + 2
    pools = model.Pools(n_pages, ps, cp, row, dtype).fill(rng)
    for slab in pools.slabs:  # scales that no append writes
        at, count = row.value_scale_offset, hkv * model.groups(row)
        slab[..., at:at + 4 * count] = rng.uniform(0.001, 3, slab.shape[:2] + (count,)).astype(np.float32).view(np.uint8).reshape(*slab.shape[:2], -1)
    slots = rng.integers(ps, (n_pages + 1) * ps, n)
    slots[::5] = np.where(rng.random(len(slots[::5])) < 0.3, -rng.integers(1, 100, len(slots[::5])), slots[::5])
    cache = cache_of(pools, dtype)
    buf = torch.full((n, hkv * (dk + dv) + 8), 7.0, dtype=dtype, device="cuda")
    k_out, v_out = buf[:, :hkv * dk].unflatten(1, (hkv, dk)), buf[:, hkv * dk:hkv * (dk + dv)].unflatten(1, (hkv, dv))
    got = cache.read_rows(torch.from_numpy(slots).cuda(), k_out=k_out, v_out=v_out)
    assert got[0] is k_out and got[1] is v_out and int(cache.d_status) == 0
    assert bool((buf[:, hkv * (dk + dv):] == 7).all())
    raw = np.stack([pools.at(max(s, ps) // ps, max(s, ps) % ps) for s in slots])
    want = [np.where((slots >= 0)[:, None, None], x, 0.0) for x in pools.rows(raw)]
    u = torch.finfo(dtype).eps / 2
    for x, y, exact in zip(got, want, (True, False)):  # keys: powers of two, or kept; values: a product in 32 bits, then rounded
        off = np.abs(x.double().cpu().numpy() - y)
        assert (off <= (0 if exact else (u + 2.0**-24) * np.abs(y)) + (0 if dtype is BF16 else 2.0**-25)).all()
    alone = cache.read_rows(torch.from_numpy(slots).cuda(), k_out=torch.empty(n, hkv, dk, dtype=dtype, device="cuda"))
    assert alone[1] is None and torch.equal(alone[0], k_out)
    both = cache.read_rows(torch.from_numpy(slots).cuda())
    assert torch.equal(both[0], k_out) and torch.equal(both[1], v_out)


def test_read_reports_bad_pages_and_clamps_fp16():
    ps, d = 4, 64
    row = QuantisedRow.of(1, d)
    pools = model.Pools(5, ps, 2, row, FP16)
    x = np.full((1, d), 65504.0)
    x[0, 1], x[0, 2] = 0.0, -65504.0
    pools.put(1, 0, x, x / 2)
    pools.at(1, 1)[:] = 0x7F  # no numbers, whatever the scale
    for slots, bit in [([4, 5, -1], 0), ([4, 5, 3], cpkv.STATUS_PAGE_OOB), ([4, 5, 24], cpkv.STATUS_PAGE_OOB), ([4, 5, 1 << 50], cpkv.STATUS_PAGE_OOB)]:
        cache = cache_of(pools, FP16)
        k, v = cache.read_rows(torch.tensor(slots).cuda())
        assert int(cache.d_status) == bit
        k, v = k.cpu(), v.cpu()
        assert not bool(k[2].any()) and not bool(v[2].any()) and bool(k[1].isnan().all()) and bool(v[1].isnan().all())
        # 65504 is nearest to 256 * 256 = 65536, which fp16 has no number for; half of it is 32768
        assert k[0, 0, 0] == 65504 and k[0, 0, 1] == 0 and k[0, 0, 2] == -65504 and v[0, 0, 0] == 32768


def test_rows_written_read_back_in_a_graph_and_on_another_stream():
    rng = np.random.default_rng(9)
    ps, d, n, hkv = 16, 64, 40, 2
    pools = model.Pools(5, ps, 2, QuantisedRow.of(hkv, d), BF16)
    cache = cache_of(pools, BF16)
    k, v = (tensor(rng.standard_normal((n, hkv, d)), BF16).cuda() for _ in range(2))
    slots = torch.from_numpy(ps + rng.permutation(5 * ps)[:n]).cuda()
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    table = torch.from_numpy(turns(rng, 4, d)).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache.append_rotary(k, v, slots, pos, table, stream=side)
    want = cache.read_rows(slots, stream=side)
    side.synchronize()
    k_out, v_out = torch.empty_like(k), torch.empty_like(v)
    cache.append_rotary(k, v, slots, pos, table)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.append_rotary(k, v, slots, pos, table)
        cache.read_rows(slots, k_out=k_out, v_out=v_out)
    for t in cache.table.pools:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(k_out, want[0]) and torch.equal(v_out, want[1]) and int(cache.d_status) == 0
    pos += 1  # new positions, the same graph
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(k_out, want[0]) and torch.equal(v_out, want[1])


def test_read_wants_its_shapes():
    pools = model.Pools(3, 16, 1, QuantisedRow.of(2, 64), BF16)
    cache = cache_of(pools, BF16)
    slots = torch.arange(16, 20).cuda()
    good = torch.empty(4, 2, 64, dtype=BF16, device="cuda")
    for bad in (good.half(), good[:3], good[:, :1], good.cpu(), good.transpose(0, 1), good[..., :32]):
        with pytest.raises(cpkv.CpkvError):
            cache.read_rows(slots, k_out=bad)
    for bad in (slots.int(), slots.cpu(), slots[::2], slots[None]):
        with pytest.raises(cpkv.CpkvError):
            cache.read_rows(bad)


@pytest.mark.parametrize("n, hq", [(3, 4), (700, 32)])
def test_append_takes_slices_and_rotates_in_place(n, hq):
    """Queries, keys and values as slices of one projection's output; the queries rotated where they stand."""
    rng = np.random.default_rng(n)
    hkv, d, ps = 2, 128, 16
    qkv = tensor(rng.standard_normal((n, hq + 2 * hkv, d)), BF16).cuda()
    pools = model.Pools(-(-n // ps) + 1, ps, 2, QuantisedRow.of(hkv, d), BF16)
    slots = torch.from_numpy(ps + rng.permutation(n)).cuda()
    table, pos = torch.from_numpy(turns(rng, 100, d)).cuda(), torch.from_numpy(rng.integers(0, 100, n).astype(np.int32)).cuda()
    one, two = cache_of(pools, BF16), cache_of(pools, BF16)
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    want = one.append_rotary(k.contiguous(), v.contiguous(), slots, pos, table, q=q.contiguous())
    two.append_rotary(k, v, slots, pos, table, q=q, q_out=q)
    assert torch.equal(q, want) and all(torch.equal(a, b) for a, b in zip(one.table.pools, two.table.pools))
    assert int(one.d_status) == 0 and int(two.d_status) == 0


def test_calls_run_with_the_pools_device_current():
    """Of a device that is not there, the switch to it fails before anything else."""
    pools = model.Pools(3, 16, 1, QuantisedRow.of(2, 64), BF16)
    cache = cache_of(pools, BF16)
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    cache.read_rows(none)
    cache.table._table.device = torch.cuda.device_count()
    rows = torch.zeros(0, 2, 64, dtype=BF16, device="cuda")
    for call in (lambda: cache.read_rows(none, k_out=rows, stream=stream),
                 lambda: cache.append_rotary(rows, rows, none, none.int(), torch.ones(8, 64, device="cuda"), stream=stream)):
        with pytest.raises(RuntimeError) as e:
            call()
        assert not isinstance(e.value, cpkv.CpkvError)
    assert torch.cuda.current_device() == 0
