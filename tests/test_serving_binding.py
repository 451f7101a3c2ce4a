"""The compiled marshalling's handling of arguments that are not what they should be (no GPU)."""
import pytest

from paged_kv_cache_compose_gb300 import build as cuda_build
from paged_kv_cache_compose_gb300 import cpkv


@pytest.fixture(scope="module")
def native():
    cuda_build.build()
    return cpkv.serving()


@pytest.mark.parametrize("call", ["append_rotary", "attend_window", "attend_shared"])
def test_tables_that_are_no_addresses(native, call):
    for table in ("table", None, -1, 1 << 70):
        with pytest.raises((TypeError, OverflowError)):
            getattr(native, call)(table, *[None] * 14)
    with pytest.raises(cpkv.CpkvError):
        getattr(native, call)(0, *[None] * 14)
    with pytest.raises(TypeError):
        getattr(native, call)(0)


def test_capture_status_of_streams(native):
    """No GPU, or the default stream: no capture; a stream that is no handle: an exception."""
    assert native.captures(0) is False
    with pytest.raises((TypeError, OverflowError)):
        native.captures("stream")
    assert cpkv.load().cpkv_stream_is_capturing(None, None) == cpkv.CPKV_ERR_ARG
