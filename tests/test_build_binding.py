"""The library's build needs neither gcc's nor Python's headers for the binding's C part, each interpreter has
its own, and without it the Python binding goes by its own checks."""
import os
import sysconfig

import pytest
import torch

import nvfp4_activation_quantize_gb300 as h3q
from nvfp4_activation_quantize_gb300 import build as libbuild


def test_the_file_is_the_interpreters():
    assert libbuild.BINDING_PATH.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


@pytest.mark.parametrize("what", ["gcc", "headers"])
def test_the_library_builds_without(what, monkeypatch, tmp_path):
    libbuild.build()
    if what == "gcc":
        monkeypatch.setattr(libbuild.shutil, "which", lambda name: None)
    else:
        monkeypatch.setattr(libbuild.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    monkeypatch.setattr(libbuild, "BINDING_PATH", str(tmp_path / "none.so"))
    assert libbuild.is_fresh()
    assert libbuild.build() == libbuild.LIB_PATH
    assert not os.path.exists(libbuild.BINDING_PATH)


def test_a_missing_binding_alone_is_built_alone(monkeypatch, tmp_path):
    libbuild.build()
    if libbuild._binding_compiler() is None:
        pytest.skip("no gcc or no Python.h")
    monkeypatch.setattr(libbuild, "BINDING_PATH", str(tmp_path / "h3q_binding.so"))
    monkeypatch.setattr(libbuild, "_nvcc", lambda: pytest.fail("the library was built again"))
    assert not libbuild.is_fresh()
    libbuild.build()
    assert os.path.exists(libbuild.BINDING_PATH) and libbuild.is_fresh()


def test_calls_without_the_module(monkeypatch, tmp_path):
    libbuild.build()
    monkeypatch.setattr(libbuild, "BINDING_PATH", str(tmp_path / "none.so"))
    monkeypatch.setattr(h3q, "_torch", None)
    monkeypatch.setattr(h3q, "_native", None)
    x, one = torch.zeros((1, 2, 64), dtype=torch.bfloat16), torch.ones(1)
    lists = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros((1, 1), dtype=torch.int32)
    cache = h3q.kv_cache_nvfp4(4, 2, 16, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA tensor"):
        h3q.h3q_kv_cache_write_nvfp4(x, x, cache, *lists, one, one)
    with pytest.raises(ValueError, match="CUDA tensor"):
        h3q.h3q_attention_cache_nvfp4(x, cache, *lists, one, one)
    with pytest.raises(ValueError, match="CUDA tensor"):
        h3q.h3q_attention_varlen(x, x, x, lists[0], lists[0])
