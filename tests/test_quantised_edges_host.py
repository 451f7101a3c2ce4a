"""Sizes of calls over quantised rows at the ends of their ranges, and the memory that a handle keeps (no GPU)."""
import weakref

import pytest

from paged_kv_cache_compose_gb300 import build as cuda_build
from paged_kv_cache_compose_gb300 import cpkv, runtime
from paged_kv_cache_compose_gb300.runtime import QuantisedCache
from test_serving_handle import attend, handle  # noqa: F401 (a fixture)


@pytest.fixture(scope="module", autouse=True)
def lib():
    cuda_build.build()


@pytest.mark.parametrize("q_lens, heads", [([1024], 32), ([256] * 3, 32), ([4000, 0], 4), ([1], 4), ([9], 8), (None, 4)], ids=str)
@pytest.mark.parametrize("window", [0, 5])
def test_no_keys_need_no_rows_read_back(q_lens, heads, window):
    """Many query rows of requests without any keys take what rows of 16 bits take: there is nothing to read back."""
    args = (len(q_lens) if q_lens else 3, heads, heads // 4, 128, q_lens, 0)
    assert cpkv.cpkv_attend_window_quantised_workspace_bytes(*args, window=window) == cpkv.cpkv_attend_window_workspace_bytes(*args, window=window)


# --------------------------------------------------------------------------- the handle's memory

@pytest.fixture
def quantised(handle, monkeypatch):
    cache = object.__new__(QuantisedCache)
    cache.__dict__.update(handle.__dict__)
    monkeypatch.setattr(QuantisedCache, "_keeps", 1000)
    return cache


class Wants:
    """A library whose attention wants `need` bytes."""

    def __init__(self, need):
        self.need, self.rooms = need, []

    def captures(self, stream):
        return False

    def attend_window(self, *args):
        self.rooms.append(None if args[12] is None else args[12].numel())
        return cpkv.CPKV_OK if args[12] is not None and args[12].numel() >= self.need else cpkv.CPKV_ERR_CAPACITY


def call(cache, need, monkeypatch):
    cache._native = Wants(need)
    monkeypatch.setattr(runtime, "_window_quantised_bytes", lambda *args: need)
    attend(cache)
    return cache._native.rooms


def test_room_for_rows_read_back_is_given_back(quantised, monkeypatch):
    """A large workspace belongs to the call: it has the size that is wanted, and the small one stays for other calls."""
    assert call(quantised, 100, monkeypatch) == [None, 125]
    assert call(quantised, 5000, monkeypatch) == [125, 5000]
    assert call(quantised, 5000, monkeypatch) == [125, 5000]
    assert call(quantised, 120, monkeypatch) == [125]
    assert call(quantised, 1000, monkeypatch) == [125, 1250]  # the most that is kept
    assert call(quantised, 1250, monkeypatch) == [1250]
    assert [w.numel() for w in quantised._workspaces.values()] == [1250]


def test_a_workspace_goes_before_a_larger_one_comes(quantised, monkeypatch):
    call(quantised, 100, monkeypatch)
    small = weakref.ref(quantised._workspaces[0, 7])
    there = []
    make = quantised._empty
    quantised._empty = lambda *args: (there.append(small() is not None), make(*args))[1]
    assert call(quantised, 500, monkeypatch) == [125, 625]
    assert there == [False] and quantised._workspaces[0, 7].numel() == 625


def test_the_gibibytes_of_a_long_prefill_are_not_kept():
    assert QuantisedCache._keeps <= 256 << 20
    assert cpkv.cpkv_attend_window_quantised_workspace_bytes(1, 32, 8, 128, [16384], 131072) > QuantisedCache._keeps
