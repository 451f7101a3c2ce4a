"""Sizes of calls over quantised rows at the ends of their ranges (no GPU)."""
import pytest

from paged_kv_cache_compose_gb300 import build as cuda_build
from paged_kv_cache_compose_gb300 import cpkv


@pytest.fixture(scope="module", autouse=True)
def lib():
    cuda_build.build()


@pytest.mark.parametrize("q_lens, heads", [([1024], 32), ([256] * 3, 32), ([4000, 0], 4), ([1], 4), ([9], 8), (None, 4)], ids=str)
@pytest.mark.parametrize("window", [0, 5])
def test_no_keys_need_no_rows_read_back(q_lens, heads, window):
    """Many query rows of requests without any keys take what rows of 16 bits take: there is nothing to read back."""
    args = (len(q_lens) if q_lens else 3, heads, heads // 4, 128, q_lens, 0)
    assert cpkv.cpkv_attend_window_quantised_workspace_bytes(*args, window=window) == cpkv.cpkv_attend_window_workspace_bytes(*args, window=window)
