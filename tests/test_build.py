"""What the C library and the calls over a bf16 cache need: not the compiled part of
the Python binding, nor torch's headers to build it against."""
import sys

import numpy as np
import pytest

import paged_kv_attention_22_gb300 as pkv
from paged_kv_attention_22_gb300 import build as pkv_build


@pytest.fixture(autouse=True)
def fresh(monkeypatch):
    pkv_build.build()
    monkeypatch.setattr(pkv, "_lib", None)
    monkeypatch.setattr(pkv, "_m", None)


def _library_works():
    assert pkv.lib().pkv_status_string(3) == b"PKV_ERR_WORKSPACE_TOO_SMALL"
    bm = pkv.BlockManager(4, 8)
    assert bm.add_sequence(0, np.arange(10, dtype=np.int32)) == 0 and bm.num_free_blocks == 2


def test_library_loads_without_the_marshalling_module(monkeypatch):
    monkeypatch.setattr(pkv, "MARSHAL_PATH", "/nonexistent/_marshal.so")
    _library_works()
    with pytest.raises(ImportError, match="/nonexistent/_marshal.so is missing"):
        pkv.kv_store_q4(None, None, None, None, None)
    _library_works()


def test_library_loads_beside_a_marshalling_module_that_does_not(monkeypatch):
    monkeypatch.delattr(pkv, "_marshal", raising=False)
    monkeypatch.setitem(sys.modules, pkv.__name__ + "._marshal", None)
    _library_works()
    with pytest.raises(ImportError):
        pkv.evict_select(None, None, 1, 0)
    _library_works()


def test_calls_of_the_marshalling_module_load_it(monkeypatch):
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        pkv.kv_store_q4(None, None, None, None, None)
    _library_works()


def test_library_is_built_without_torch(monkeypatch):
    def no_torch():
        raise ImportError("no torch here")
    monkeypatch.setattr(pkv_build, "_torch", no_torch)
    assert pkv_build.build_library() == pkv_build.LIBRARY
    # with something to build for each: the library is there before the failure
    linked = []
    monkeypatch.setattr(pkv_build, "_library_stale", lambda: True)
    monkeypatch.setattr(pkv_build, "_marshal_stale", lambda: True)
    monkeypatch.setattr(pkv_build, "SOURCES", ["block_manager.cpp"])
    monkeypatch.setattr(pkv_build, "_link", lambda cmd, target: linked.append(target))
    with pytest.raises(ImportError, match="no torch here"):
        pkv_build.build()
    assert linked == [pkv_build.LIBRARY]
