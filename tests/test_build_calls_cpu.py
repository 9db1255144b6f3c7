"""The extension module of the Python calls belongs to one torch, one C++ ABI and one interpreter:
it is built anew, under another name, for any other."""
import os
import sysconfig

import torch

import speculative_decoding_drafter_head_b200 as ds
from speculative_decoding_drafter_head_b200 import _build


def test_the_file_names_what_it_was_built_for():
    name = os.path.basename(_build.calls_path())
    assert torch.__version__ in name and sysconfig.get_config_var("EXT_SUFFIX") in name
    assert f"abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)}" in name
    assert os.path.dirname(_build.calls_path()) == _build.PKG


def test_another_torch_or_interpreter_makes_it_stale(monkeypatch):
    ds.calls()
    assert not _build.calls_stale()
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1+other")
        assert _build.calls_stale()
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
        assert _build.calls_stale()
    with monkeypatch.context() as m:
        get = sysconfig.get_config_var
        m.setattr(sysconfig, "get_config_var",
                  lambda k: ".cpython-399-none.so" if k == "EXT_SUFFIX" else get(k))
        assert _build.calls_stale()
    assert not _build.calls_stale()
