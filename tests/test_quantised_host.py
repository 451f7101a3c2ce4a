"""Quantised rows on the host: the model of their format, layouts, refusals before anything is launched (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

import quantised_model as model
from paged_kv_cache_compose_gb300 import build as cuda_build
from paged_kv_cache_compose_gb300 import cpkv
from paged_kv_cache_compose_gb300.cpkv import QuantisedRow
from paged_kv_cache_compose_gb300.runtime import QuantisedCache
from test_serving_host import FAKE, Args, pools


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return cpkv.load()


def test_the_model_knows_e4m3():
    """torch's conversion, an independent one, agrees with the model's table and rounding."""
    assert np.array_equal(model.VALUES, torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    rng = np.random.default_rng(0)
    y = np.concatenate([rng.uniform(-448, 448, 4000), rng.uniform(-0.02, 0.02, 4000), (model.VALUES[:126] + model.VALUES[1:127]) / 2, [0.0, -0.0]])
    y = y.astype(np.float32).astype(np.float64)
    assert np.array_equal(model.to_e4m3(y), torch.from_numpy(y).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_scales_are_the_smallest_powers():
    x = np.array([[448.0], [448.1], [0.0], [1.75], [1.76], [3e38], [np.inf], [2.0**-140]])
    assert model.scale_of(x).tolist() == [1.0, 2.0, 2.0**-126, 2.0**-8, 2.0**-7, 2.0**120, 2.0**-126, 2.0**-126]


@pytest.mark.parametrize("args, size", [((8, 128), 2112), ((8, 64), 1088), ((1, 64), 144), ((1, 64, 512, True), 656), ((1, 128, 256), 400), ((3, 64, 128, True), 784)])
def test_row_layouts(args, size):
    row = QuantisedRow.of(*args)
    assert row.row_bytes == size == QuantisedCache.row_bytes(*args)
    parts = [(row.value_offset, row.kv_heads * row.value_dim), (row.value_scale_offset, 4 * row.kv_heads * model.groups(row)),
             (row.key_offset, row.kv_heads * row.key_dim * (2 if row.keep_keys else 1))]
    if not row.keep_keys:
        parts.append((row.key_scale_offset, 4 * row.kv_heads))
    parts.sort()
    assert all(a + n <= b for (a, n), (b, _) in zip(parts, parts[1:])) and parts[-1][0] + parts[-1][1] <= row.row_bytes


def row_of(base=None, **changed):
    row = base or QuantisedRow.of(2, 64)
    for name, value in changed.items():
        setattr(row, name, value)
    return row


BAD_ROWS = [(dict(kv_heads=0), cpkv.CPKV_ERR_ARG), (dict(kv_heads=1025), cpkv.CPKV_ERR_LIMIT), (dict(key_dim=96), cpkv.CPKV_ERR_LIMIT),
            (dict(key_dim=0), cpkv.CPKV_ERR_ARG), (dict(value_dim=192), cpkv.CPKV_ERR_LIMIT), (dict(value_dim=32), cpkv.CPKV_ERR_LIMIT),
            (dict(value_dim=8192), cpkv.CPKV_ERR_LIMIT), (dict(key_offset=8), cpkv.CPKV_ERR_ARG), (dict(key_offset=-16), cpkv.CPKV_ERR_ARG),
            (dict(value_offset=64), cpkv.CPKV_ERR_ARG), (dict(value_offset=160), cpkv.CPKV_ERR_ARG), (dict(key_scale_offset=258), cpkv.CPKV_ERR_ARG),
            (dict(key_scale_offset=128), cpkv.CPKV_ERR_ARG), (dict(value_scale_offset=268), cpkv.CPKV_ERR_ARG),
            (dict(value_scale_offset=260), cpkv.CPKV_ERR_ARG), (dict(key_offset=2**62), cpkv.CPKV_ERR_ARG), (dict(row_bytes=264), cpkv.CPKV_ERR_ARG),
            (dict(row_bytes=256), cpkv.CPKV_ERR_ARG), (dict(keep_keys=1), cpkv.CPKV_ERR_ARG), (dict(keep_keys=1, key_dim=4), cpkv.CPKV_ERR_LIMIT)]


class Row:
    """A row as an argument that stays alive."""

    def __init__(self, row):
        self.row = row

    def __repr__(self):
        return "row"


def call(args, fn, **changed):
    changed = {k: ctypes.addressof(v.row) if isinstance(v, Row) else v for k, v in {**args, **changed}.items()}
    return Args(changed)(fn)


def append_args():
    return Args(n=3, ps=16, cp=2, dtype=cpkv.BF16, hq=4, row=Row(row_of()), pools=pools(), caps=np.array([4, 4], np.int64), k=FAKE, ks=128,
                v=FAKE, vs=128, q=FAKE, qs=256, qo=FAKE, qos=256, slots=FAKE, pos=FAKE, pos_stride=3, axes=1, axis=None, table=FAKE, max_pos=100,
                rot=64, flags=0, status=FAKE, stream=None)


@pytest.mark.parametrize("changed, code", [
    (dict(n=0), cpkv.CPKV_OK), (dict(n=-1), cpkv.CPKV_ERR_ARG), (dict(n=1 << 31), cpkv.CPKV_ERR_LIMIT), (dict(ps=0), cpkv.CPKV_ERR_ARG),
    (dict(cp=65), cpkv.CPKV_ERR_LIMIT), (dict(dtype=2), cpkv.CPKV_ERR_ARG), (dict(hq=-1), cpkv.CPKV_ERR_ARG), (dict(row=None), cpkv.CPKV_ERR_ARG),
    (dict(rot=24), cpkv.CPKV_ERR_ARG), (dict(rot=80), cpkv.CPKV_ERR_ARG), (dict(pools=pools(address=264)), cpkv.CPKV_ERR_ARG),
    (dict(k=None), cpkv.CPKV_ERR_ARG), (dict(v=264), cpkv.CPKV_ERR_ARG), (dict(ks=120), cpkv.CPKV_ERR_ARG), (dict(vs=132), cpkv.CPKV_ERR_ARG),
    (dict(q=None), cpkv.CPKV_ERR_ARG), (dict(qos=248), cpkv.CPKV_ERR_ARG), (dict(slots=None), cpkv.CPKV_ERR_ARG), (dict(axes=5), cpkv.CPKV_ERR_ARG),
    (dict(axes=3), cpkv.CPKV_ERR_ARG), (dict(axes=3, axis=np.full(32, 3, np.uint8)), cpkv.CPKV_ERR_ARG), (dict(table=None), cpkv.CPKV_ERR_ARG),
    (dict(max_pos=0), cpkv.CPKV_ERR_ARG), (dict(flags=1), cpkv.CPKV_ERR_ARG), (dict(status=None), cpkv.CPKV_ERR_ARG),
] + [(dict(row=Row(row_of(**bad))), code) for bad, code in BAD_ROWS], ids=str)
def test_append_refusals(lib, changed, code):
    assert call(append_args(), lib.cpkv_append_quantised, **changed) == code


def read_args():
    return Args(n=3, ps=16, cp=2, dtype=cpkv.BF16, row=Row(row_of()), pools=pools(), caps=np.array([4, 4], np.int64), slots=FAKE, k=FAKE, ks=128,
                v=FAKE, vs=128, flags=0, status=FAKE, stream=None)


@pytest.mark.parametrize("changed, code", [
    (dict(n=0), cpkv.CPKV_OK), (dict(n=0, k=None, v=None), cpkv.CPKV_OK), (dict(n=-1), cpkv.CPKV_ERR_ARG), (dict(n=1 << 31), cpkv.CPKV_ERR_LIMIT),
    (dict(ps=0), cpkv.CPKV_ERR_ARG), (dict(cp=0), cpkv.CPKV_ERR_ARG), (dict(dtype=2), cpkv.CPKV_ERR_ARG), (dict(row=None), cpkv.CPKV_ERR_ARG),
    (dict(pools=None), cpkv.CPKV_ERR_ARG), (dict(slots=None), cpkv.CPKV_ERR_ARG), (dict(k=None, v=None), cpkv.CPKV_ERR_ARG),
    (dict(k=264), cpkv.CPKV_ERR_ARG), (dict(v=260), cpkv.CPKV_ERR_ARG), (dict(ks=120), cpkv.CPKV_ERR_ARG), (dict(vs=130), cpkv.CPKV_ERR_ARG),
    (dict(flags=8), cpkv.CPKV_ERR_ARG), (dict(status=None), cpkv.CPKV_ERR_ARG),
] + [(dict(row=Row(row_of(**bad))), code) for bad, code in BAD_ROWS], ids=str)
def test_read_refusals(lib, changed, code):
    assert call(read_args(), lib.cpkv_read_quantised, **changed) == code


def test_tables_want_byte_pools_of_whole_rows():
    row = QuantisedRow.of(2, 64)
    good = torch.zeros(3, 16, row.row_bytes, dtype=torch.uint8)
    for bad, ps, dtype in (([good.half()], 16, torch.bfloat16), ([good[:, :, :256].contiguous()], 16, torch.bfloat16), ([good], 8, torch.bfloat16),
                           ([good], 16, torch.float32), ([], 16, torch.bfloat16), ([good], 16, torch.bfloat16)):  # the last: host memory
        with pytest.raises(cpkv.CpkvError):
            cpkv.QuantisedTable(bad, ps, row, dtype)
    with pytest.raises(cpkv.CpkvError):  # a row of other heads
        QuantisedCache([good], page_size=16, kv_heads=1, key_dim=64, row=row)


def window_args():
    return Args(B=2, ps=16, cp=2, dtype=cpkv.BF16, hq=4, row=Row(row_of()), q_lens=np.array([1, 2], np.int32), max_kv=64, pools=pools(),
                caps=np.array([4, 4], np.int64), table=FAKE, stride=4, kv_lens=FAKE, tokens=3, q=FAKE, qs=256, scale=0.1, window=8, sinks=2, out=FAKE,
                os=256, lse=None, ws=FAKE, ws_bytes=1 << 40, flags=0, status=FAKE, stream=None)


def shared_args():
    return Args(B=3, groups=2, ps=16, cp=2, dtype=cpkv.FP16, hq=4, row=Row(row_of()), sizes=np.array([1, 2], np.int32),
                prefix=np.array([32, 0], np.int32), max_suffix=64, pools=pools(), caps=np.array([4, 4], np.int64), prefix_pages=FAKE, n_prefix=2,
                table=FAKE, stride=4, suffix=FAKE, q=FAKE, qs=256, scale=0.1, out=FAKE, os=256, lse=None, ws=FAKE, ws_bytes=1 << 40, flags=0,
                status=FAKE, stream=None)


UNFIT = [(dict(row=Row(QuantisedRow.of(1, 64, 512, True))), cpkv.CPKV_ERR_ARG), (dict(row=Row(QuantisedRow.of(1, 64, 128))), cpkv.CPKV_ERR_ARG),
         (dict(row=None), cpkv.CPKV_ERR_ARG), (dict(hq=3), cpkv.CPKV_ERR_ARG), (dict(hq=4100), cpkv.CPKV_ERR_LIMIT), (dict(dtype=5), cpkv.CPKV_ERR_ARG),
         (dict(q=None), cpkv.CPKV_ERR_ARG), (dict(q=260), cpkv.CPKV_ERR_ARG), (dict(out=None), cpkv.CPKV_ERR_ARG), (dict(os=128), cpkv.CPKV_ERR_ARG),
         (dict(scale=float("nan")), cpkv.CPKV_ERR_ARG), (dict(ws_bytes=16), cpkv.CPKV_ERR_CAPACITY), (dict(ws=264), cpkv.CPKV_ERR_ARG),
         (dict(flags=1), cpkv.CPKV_ERR_ARG), (dict(status=None), cpkv.CPKV_ERR_ARG), (dict(table=None), cpkv.CPKV_ERR_ARG),
         (dict(pools=None), cpkv.CPKV_ERR_ARG), (dict(stride=-1), cpkv.CPKV_ERR_CAPACITY)] + [(dict(row=Row(row_of(**bad))), code) for bad, code in BAD_ROWS]


@pytest.mark.parametrize("changed, code", UNFIT + [
    (dict(B=0, tokens=0), cpkv.CPKV_OK), (dict(tokens=4), cpkv.CPKV_ERR_ARG), (dict(max_kv=65), cpkv.CPKV_ERR_CAPACITY),
    (dict(window=-1), cpkv.CPKV_ERR_ARG), (dict(sinks=-1), cpkv.CPKV_ERR_ARG), (dict(kv_lens=None), cpkv.CPKV_ERR_ARG)], ids=str)
def test_window_refusals(lib, changed, code):
    assert call(window_args(), lib.cpkv_attend_window_quantised, **changed) == code


@pytest.mark.parametrize("changed, code", UNFIT + [
    (dict(B=0, groups=0), cpkv.CPKV_OK), (dict(B=2), cpkv.CPKV_ERR_ARG), (dict(prefix=np.array([31, 0], np.int32)), cpkv.CPKV_ERR_UNALIGNED_PREFIX),
    (dict(n_prefix=1), cpkv.CPKV_ERR_CAPACITY), (dict(max_suffix=65), cpkv.CPKV_ERR_CAPACITY), (dict(suffix=None), cpkv.CPKV_ERR_ARG)], ids=str)
def test_shared_refusals(lib, changed, code):
    assert call(shared_args(), lib.cpkv_attend_shared_quantised, **changed) == code


def test_workspace_sizes(lib):
    """Many query rows: room for the rows that they see, in 16 bits, as far as a window lets them see; never more than 4 GiB of it."""
    def size(*args, **more):
        return cpkv.cpkv_attend_window_quantised_workspace_bytes(*args, **more)

    def plain(*args, **more):
        return cpkv.cpkv_attend_window_workspace_bytes(*args, **more)

    for few in ((1, 4, 1, 64, None, 100), (64, 32, 8, 128, None, 100_000), (3, 32, 8, 128, [100, 100, 100], 5000)):
        assert size(*few) == plain(*few)
    many = (2, 32, 8, 128, [400, 300], 20_000)
    rows = 2 * -(-20_000 // 32) * 32 * 8 * 128 * 4
    assert rows <= size(*many) - plain(*many) <= rows + (1 << 20)
    assert size(*many, window=512) - plain(*many, window=512) <= (2 * (512 + 400 + 64 + 96)) * 8 * 128 * 4
    huge = (64, 32, 8, 128, [400] * 64, 1_000_000)
    assert size(*huge) == plain(*huge)
    for bad in (dict(head_dim=96), dict(B=1025), dict(q_heads=3), dict(window=-1), dict(max_kv_len=-1)):
        args = dict(B=1, q_heads=4, kv_heads=2, head_dim=64, q_lens=None, max_kv_len=10)
        with pytest.raises(cpkv.CpkvError):
            size(**{**args, **bad})


def test_shared_workspace_sizes(lib):
    """Suffixes beside prefixes of many rows have parts of their own; few rows need what plain rows do."""
    def size(*args, **named):
        return cpkv.cpkv_attend_shared_quantised_workspace_bytes(*args, **named)

    def plain(*args):
        return cpkv.cpkv_attend_shared_workspace_bytes(*args)

    for same in ((4, 8, 2, 128, [1, 3], [64, 0], 50), (1, 4, 2, 64, [1], [100], 10), (40, 64, 2, 64, [40], [512], 300)):
        assert size(*same) == plain(*same)
    assert size(64, 32, 8, 128, [64], [4096], 1024) > 64 * 8 * 16 * 129 * 4  # a part of 16 rows for each request and head
    assert size(0, 8, 2, 128, [], [], 0) >= 0
    for changed in (dict(head_dim=96), dict(B=1025), dict(B=3), dict(q_heads=3), dict(max_suffix_len=-1), dict(prefix_lens=[-16])):
        args = dict(B=2, q_heads=4, kv_heads=2, head_dim=64, group_sizes=[2], prefix_lens=[16], max_suffix_len=10)
        with pytest.raises(cpkv.CpkvError):
            size(**{**args, **changed})
    assert lib.cpkv_attend_shared_quantised_workspace_bytes(1, 1, 4, 2, 64, None, None, 10, ctypes.byref(ctypes.c_int64())) == cpkv.CPKV_ERR_ARG
