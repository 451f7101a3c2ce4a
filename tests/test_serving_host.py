"""Refusals and sizes of the serving calls, before anything is launched (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_cache_compose_gb300 import build as cuda_build
from paged_kv_cache_compose_gb300 import cpkv

FAKE = 256  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return cpkv.load()


class Args(dict):
    def __call__(self, fn, **changed):
        keep = []
        values = []
        for key, value in {**self, **changed}.items():
            if isinstance(value, np.ndarray):
                keep.append(value)
                value = value.ctypes.data
            values.append(value)
        assert not set(changed) - set(self), changed
        return fn(*values)


def pools(n=2, address=FAKE):
    return np.full(n, address, np.uint64)


def append_args():
    return Args(n=3, ps=16, cp=2, dtype=cpkv.BF16, hq=4, hkv=2, dk=64, dv=64, row=512, k_off=0, v_off=256, pools=pools(),
                caps=np.array([4, 4], np.int64), k=FAKE, ks=128, v=FAKE, vs=128, q=FAKE, qs=256, qo=FAKE, qos=256, slots=FAKE, pos=FAKE,
                pos_stride=3, axes=1, axis=None, table=FAKE, max_pos=100, rot=64, flags=0, status=FAKE, stream=None)


@pytest.mark.parametrize("changed, code", [
    (dict(n=0), cpkv.CPKV_OK),
    (dict(n=-1), cpkv.CPKV_ERR_ARG), (dict(ps=0), cpkv.CPKV_ERR_ARG), (dict(cp=0), cpkv.CPKV_ERR_ARG), (dict(cp=65), cpkv.CPKV_ERR_LIMIT),
    (dict(dtype=2), cpkv.CPKV_ERR_ARG), (dict(hkv=0), cpkv.CPKV_ERR_ARG), (dict(hq=-1), cpkv.CPKV_ERR_ARG),
    (dict(dk=60), cpkv.CPKV_ERR_ARG), (dict(dv=4), cpkv.CPKV_ERR_ARG), (dict(rot=24), cpkv.CPKV_ERR_ARG), (dict(rot=80), cpkv.CPKV_ERR_ARG),
    (dict(row=520), cpkv.CPKV_ERR_ARG), (dict(row=496), cpkv.CPKV_ERR_ARG), (dict(v_off=128), cpkv.CPKV_ERR_ARG),
    (dict(v_off=264), cpkv.CPKV_ERR_ARG), (dict(k_off=-16), cpkv.CPKV_ERR_ARG), (dict(pools=None), cpkv.CPKV_ERR_ARG),
    (dict(pools=pools(address=0)), cpkv.CPKV_ERR_ARG), (dict(pools=pools(address=264)), cpkv.CPKV_ERR_ARG),
    (dict(caps=np.array([4, -1], np.int64)), cpkv.CPKV_ERR_ARG), (dict(k=None), cpkv.CPKV_ERR_ARG), (dict(v=264), cpkv.CPKV_ERR_ARG),
    (dict(ks=120), cpkv.CPKV_ERR_ARG), (dict(vs=132), cpkv.CPKV_ERR_ARG), (dict(q=None), cpkv.CPKV_ERR_ARG), (dict(qo=None), cpkv.CPKV_ERR_ARG),
    (dict(qs=248), cpkv.CPKV_ERR_ARG), (dict(slots=None), cpkv.CPKV_ERR_ARG), (dict(pos=None), cpkv.CPKV_ERR_ARG),
    (dict(axes=0), cpkv.CPKV_ERR_ARG), (dict(axes=5), cpkv.CPKV_ERR_ARG), (dict(axes=3), cpkv.CPKV_ERR_ARG),
    (dict(axes=3, axis=np.full(32, 3, np.uint8)), cpkv.CPKV_ERR_ARG), (dict(axes=3, axis=np.zeros(32, np.uint8), pos_stride=2), cpkv.CPKV_ERR_ARG),
    (dict(table=None), cpkv.CPKV_ERR_ARG), (dict(table=264), cpkv.CPKV_ERR_ARG), (dict(max_pos=0), cpkv.CPKV_ERR_ARG),
    (dict(max_pos=1 << 40), cpkv.CPKV_ERR_LIMIT), (dict(flags=1), cpkv.CPKV_ERR_ARG), (dict(status=None), cpkv.CPKV_ERR_ARG),
    (dict(n=1 << 31), cpkv.CPKV_ERR_LIMIT),
], ids=str)
def test_append_refusals(lib, changed, code):
    assert append_args()(lib.cpkv_append_rotary, **changed) == code


def window_args():
    return Args(B=2, ps=16, cp=2, dtype=cpkv.BF16, hq=4, hkv=2, d=64, row=512, k_off=0, v_off=256, q_lens=np.array([1, 2], np.int32),
                max_kv=64, pools=pools(), caps=np.array([4, 4], np.int64), table=FAKE, stride=4, kv_lens=FAKE, tokens=3, q=FAKE, qs=256, scale=0.1,
                window=8, sinks=2, out=FAKE, os=256, lse=None, ws=FAKE, ws_bytes=1 << 40, flags=0, status=FAKE, stream=None)


@pytest.mark.parametrize("changed, code", [
    (dict(B=0, tokens=0), cpkv.CPKV_OK), (dict(q_lens=np.zeros(2, np.int32), tokens=0), cpkv.CPKV_OK),
    (dict(tokens=4), cpkv.CPKV_ERR_ARG), (dict(tokens=0), cpkv.CPKV_ERR_ARG),
    (dict(B=-1), cpkv.CPKV_ERR_ARG), (dict(B=1025, q_lens=None), cpkv.CPKV_ERR_LIMIT), (dict(q_lens=np.array([1, -1], np.int32)), cpkv.CPKV_ERR_ARG),
    (dict(ps=-4), cpkv.CPKV_ERR_ARG), (dict(dtype=5), cpkv.CPKV_ERR_ARG), (dict(hq=3), cpkv.CPKV_ERR_ARG), (dict(hkv=0), cpkv.CPKV_ERR_ARG), (dict(hq=4100), cpkv.CPKV_ERR_LIMIT),
    (dict(hq=1025, hkv=1025), cpkv.CPKV_ERR_LIMIT), (dict(d=96), cpkv.CPKV_ERR_LIMIT), (dict(d=128), cpkv.CPKV_ERR_ARG), (dict(max_kv=-1), cpkv.CPKV_ERR_ARG),
    (dict(max_kv=65), cpkv.CPKV_ERR_CAPACITY), (dict(stride=-1), cpkv.CPKV_ERR_CAPACITY), (dict(window=-1), cpkv.CPKV_ERR_ARG),
    (dict(sinks=-1), cpkv.CPKV_ERR_ARG), (dict(table=None), cpkv.CPKV_ERR_ARG), (dict(kv_lens=None), cpkv.CPKV_ERR_ARG),
    (dict(q=None), cpkv.CPKV_ERR_ARG), (dict(q=260), cpkv.CPKV_ERR_ARG), (dict(qs=252), cpkv.CPKV_ERR_ARG), (dict(os=128), cpkv.CPKV_ERR_ARG),
    (dict(out=None), cpkv.CPKV_ERR_ARG), (dict(scale=float("nan")), cpkv.CPKV_ERR_ARG), (dict(scale=float("inf")), cpkv.CPKV_ERR_ARG),
    (dict(ws=None), cpkv.CPKV_ERR_ARG), (dict(ws=264), cpkv.CPKV_ERR_ARG), (dict(ws_bytes=16), cpkv.CPKV_ERR_CAPACITY),
    (dict(ws=None, ws_bytes=0), cpkv.CPKV_ERR_CAPACITY), (dict(flags=1), cpkv.CPKV_ERR_ARG), (dict(status=None), cpkv.CPKV_ERR_ARG), (dict(v_off=264), cpkv.CPKV_ERR_ARG),
    (dict(k_off=272), cpkv.CPKV_ERR_ARG), (dict(pools=None), cpkv.CPKV_ERR_ARG),
], ids=str)
def test_window_refusals(lib, changed, code):
    assert window_args()(lib.cpkv_attend_window, **changed) == code


def shared_args():
    return Args(B=3, groups=2, ps=16, cp=2, dtype=cpkv.FP16, hq=4, hkv=2, d=64, row=512, k_off=0, v_off=256, sizes=np.array([1, 2], np.int32),
                prefix=np.array([32, 0], np.int32), max_suffix=64, pools=pools(), caps=np.array([4, 4], np.int64), prefix_pages=FAKE, n_prefix=2,
                table=FAKE, stride=4, suffix=FAKE, q=FAKE, qs=256, scale=0.1, out=FAKE, os=256, lse=None, ws=FAKE, ws_bytes=1 << 40, flags=0,
                status=FAKE, stream=None)


@pytest.mark.parametrize("changed, code", [
    (dict(B=0, groups=0), cpkv.CPKV_OK), (dict(B=2), cpkv.CPKV_ERR_ARG), (dict(groups=1), cpkv.CPKV_ERR_ARG), (dict(groups=-1), cpkv.CPKV_ERR_ARG),
    (dict(sizes=None), cpkv.CPKV_ERR_ARG), (dict(sizes=np.array([4, -1], np.int32)), cpkv.CPKV_ERR_ARG),
    (dict(prefix=np.array([31, 0], np.int32)), cpkv.CPKV_ERR_UNALIGNED_PREFIX), (dict(prefix=np.array([-16, 0], np.int32)), cpkv.CPKV_ERR_ARG),
    (dict(prefix_pages=None), cpkv.CPKV_ERR_ARG), (dict(n_prefix=1), cpkv.CPKV_ERR_CAPACITY), (dict(max_suffix=65), cpkv.CPKV_ERR_CAPACITY), (dict(d=80), cpkv.CPKV_ERR_LIMIT),
    (dict(suffix=None), cpkv.CPKV_ERR_ARG), (dict(ws_bytes=64), cpkv.CPKV_ERR_CAPACITY), (dict(ws=None), cpkv.CPKV_ERR_ARG),
    (dict(flags=8), cpkv.CPKV_ERR_ARG), (dict(status=None), cpkv.CPKV_ERR_ARG), (dict(q=None), cpkv.CPKV_ERR_ARG),
    (dict(B=1025, sizes=np.array([1024, 1], np.int32)), cpkv.CPKV_ERR_LIMIT), (dict(hq=5), cpkv.CPKV_ERR_ARG),
], ids=str)
def test_shared_refusals(lib, changed, code):
    assert shared_args()(lib.cpkv_attend_shared, **changed) == code


def test_workspace_sizes(lib):
    small = cpkv.cpkv_attend_window_workspace_bytes(1, 4, 1, 64, None, 100)
    assert small == 0  # few keys: whole tiles, nothing to join
    assert 0 < cpkv.cpkv_attend_window_workspace_bytes(64, 32, 8, 128, None, 100_000)
    # a window bounds the work of long requests, and so the workspace
    assert cpkv.cpkv_attend_window_workspace_bytes(1, 4, 1, 64, None, 100_000, window=256) < \
        cpkv.cpkv_attend_window_workspace_bytes(1, 4, 1, 64, None, 100_000)
    assert cpkv.cpkv_attend_shared_workspace_bytes(4, 8, 2, 128, [1, 3], [64, 0], 50) > 0
    for bad in (dict(head_dim=96), dict(B=1025), dict(q_heads=3)):
        args = dict(B=1, q_heads=4, kv_heads=2, head_dim=64, q_lens=None, max_kv_len=10)
        with pytest.raises(cpkv.CpkvError):
            cpkv.cpkv_attend_window_workspace_bytes(**{**args, **bad})
    out = ctypes.c_int64(0)
    assert lib.cpkv_attend_window_workspace_bytes(1, 4, 2, 64, None, 10, -1, 0, ctypes.byref(out)) == cpkv.CPKV_ERR_ARG
    assert lib.cpkv_attend_shared_workspace_bytes(1, 1, 4, 2, 64, None, None, 10, ctypes.byref(out)) == cpkv.CPKV_ERR_ARG


def test_pool_table_wants_paged_pools():
    good = torch.zeros(3, 16, 256, dtype=torch.bfloat16)
    for pools_, ps in (([], 16), ([good.float()], 16), ([good], 8), ([good, good[:, :, :128]], 16), ([good, good.half()], 16),
                       ([good.flatten(1)], 16)):
        with pytest.raises(cpkv.CpkvError):
            cpkv.PoolTable(pools_, ps, 0, 256)
    with pytest.raises(cpkv.CpkvError):  # host memory
        cpkv.PoolTable([good], 16, 0, 256)
