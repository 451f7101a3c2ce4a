"""The serving handle's host logic with the compiled calls replaced (no GPU)."""
import contextlib
import types

import pytest
import torch

from paged_kv_cache_compose_gb300 import build as cuda_build
from paged_kv_cache_compose_gb300 import cpkv, runtime
from paged_kv_cache_compose_gb300.runtime import PagedCache

NEED = 1000


class Native:
    """A library whose attention wants NEED bytes; `during` runs inside its first call."""

    def __init__(self, during=lambda: None, captured=False):
        self.rooms, self.during, self.captured = [], during, captured

    def captures(self, stream):
        return self.captured

    def attend_window(self, *args):
        room = args[12]
        self.rooms.append(room)
        if len(self.rooms) == 1:
            self.during()
        return cpkv.CPKV_OK if room is not None and room.numel() >= NEED else cpkv.CPKV_ERR_CAPACITY


@pytest.fixture
def handle(monkeypatch):
    cuda_build.build()
    cache = object.__new__(PagedCache)
    cache.kv_heads = cache.key_dim = cache.value_dim = 64
    cache.table, cache.device, cache.d_status, cache._scale = types.SimpleNamespace(native=0), torch.device("cuda", 0), None, 1.0
    monkeypatch.setattr(PagedCache, "_workspaces", {})
    cache._stream = lambda stream: 7
    cache._empty = lambda shape, dtype, stream: torch.empty(shape, dtype=dtype)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(runtime, "_window_bytes", lambda *args: NEED)
    return cache


def attend(cache, **more):
    q = torch.zeros(1, 1, 64)
    return cache.attend_window(q, None, None, None, max_kv_len=1, out=q, **more)


def test_the_workspace_grows_once_and_stays(handle):
    handle._native = Native()
    attend(handle)
    attend(handle)
    first, grown, again = handle._native.rooms
    assert first is None and grown.numel() >= NEED and again is grown


def test_a_workspace_that_another_thread_grew_meanwhile(handle):
    """Another thread replaces the workspace between this call's failure and its look at the size: the call still runs."""
    def other():
        handle._workspaces[0, 7] = torch.empty(2 * NEED, dtype=torch.uint8)

    handle._native = Native(other)
    attend(handle)
    assert handle._native.rooms[-1].numel() >= NEED


def test_a_capacity_that_no_workspace_mends(handle, monkeypatch):
    """A call that fails for another capacity (its page table's) is refused, not tried again and again."""
    handle._native = Native()
    monkeypatch.setattr(runtime, "_window_bytes", lambda *args: 0)
    with pytest.raises(cpkv.CpkvError):
        attend(handle)
    assert len(handle._native.rooms) == 1


def test_captured_calls_keep_nothing(handle):
    handle._native = Native(captured=True)
    attend(handle)
    attend(handle)
    assert not handle._workspaces and [r is None for r in handle._native.rooms] == [True, False, True, False]


def test_a_workspace_of_the_caller_is_not_replaced(handle):
    handle._native = Native()
    with pytest.raises(cpkv.CpkvError):
        attend(handle, workspace=torch.empty(NEED - 1, dtype=torch.uint8))
    assert len(handle._native.rooms) == 1 and not handle._workspaces


def test_handles_share_the_workspace_of_a_stream(handle):
    """A model's layers, one handle each, keep one workspace and not one each."""
    other = object.__new__(PagedCache)
    other.__dict__.update(handle.__dict__)
    handle._native, other._native = Native(), Native()
    attend(handle)
    attend(other)
    assert other._native.rooms == [handle._native.rooms[-1]]
