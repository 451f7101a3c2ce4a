"""Sizes of the serving calls at their limits, before anything is launched (no GPU)."""
import pytest

from paged_kv_cache_compose_gb300 import build as cuda_build
from paged_kv_cache_compose_gb300 import cpkv


@pytest.fixture(scope="module", autouse=True)
def lib():
    cuda_build.build()
    return cpkv.load()


@pytest.mark.parametrize("prefix, fits", [(2**30 - 16, True), (2**30, False), (2**31 - 16, False)])
def test_prefixes_past_30_bits_are_refused(prefix, fits):
    """Key positions of a prefix, rounded up to a tile, stay in 32 bits."""
    def size():
        return cpkv.cpkv_attend_shared_workspace_bytes(1, 4, 2, 64, [1], [prefix], 10)

    if fits:
        assert size() > 0
    else:
        with pytest.raises(cpkv.CpkvError) as e:
            size()
        assert e.value.code == cpkv.CPKV_ERR_LIMIT


@pytest.mark.parametrize("q_lens", [None, [3, 3], [40, 2]])
def test_a_window_past_the_longest_request_is_none(q_lens):
    sizes = {cpkv.cpkv_attend_window_workspace_bytes(2, 8, 2, 64, q_lens, 5000, window=w) for w in (0, 5000, 5001, 2**31 - 1)}
    assert len(sizes) == 1
