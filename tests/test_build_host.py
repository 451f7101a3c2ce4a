"""When the marshalling of the serving calls is built, and for what (no GPU)."""
import sys
import sysconfig
import types

import pytest

import paged_kv_cache_compose_gb300 as package
from paged_kv_cache_compose_gb300 import build as cuda_build
from paged_kv_cache_compose_gb300 import cpkv


@pytest.fixture(autouse=True)
def built():
    cuda_build.build()


def test_nothing_is_stale_after_a_build():
    assert not cuda_build.stale() and not cuda_build.binding_stale()
    assert cuda_build.BINDING_PATH.endswith(sysconfig.get_config_var("EXT_SUFFIX"))  # another Python does not load it


def test_the_library_is_built_without_torch(monkeypatch):
    """Where torch is missing the build ends well without the marshalling, which the compose does not use."""
    def wanted(*args):
        raise AssertionError("the marshalling is not to be built")

    monkeypatch.setattr(cuda_build, "torch_version", lambda: None)
    monkeypatch.setattr(cuda_build, "BINDING_PATH", "/nowhere/_serving.so")
    monkeypatch.setattr(cuda_build, "_compile_binding", wanted)
    assert cuda_build.build() == cuda_build.LIB_PATH


def test_another_torch_makes_it_stale(monkeypatch):
    monkeypatch.setattr(cuda_build, "torch_version", lambda: "0.1")
    assert cuda_build.binding_stale()


def test_one_built_for_another_torch_is_not_used(monkeypatch):
    other = types.SimpleNamespace(built_for="0.1", set_fail=lambda f: None)
    monkeypatch.setitem(sys.modules, package.__name__ + "._serving", other)
    monkeypatch.setattr(package, "_serving", other, raising=False)
    monkeypatch.setattr(cpkv, "_native", None)
    with pytest.raises(cpkv.CpkvError, match="0.1"):
        cpkv.serving()
