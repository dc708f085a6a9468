"""The in-tree build: what is built without what, and what counts as stale.  In a
folder of its own, with a source of one line in place of the library's."""
import os
import sysconfig

import pytest
import torch

from gated_deltanet_prefill_gb300 import attn
from gated_deltanet_prefill_gb300 import build as gbuild


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    source = tmp_path / "one.cu"
    source.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(gbuild, "sources", lambda: [str(source)])
    monkeypatch.setattr(gbuild, "BUILD", str(tmp_path))
    monkeypatch.setattr(gbuild, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(gbuild, "_stale", lambda lib=None: not os.path.exists(gbuild.LIB))
    return tmp_path


def test_library_is_linked_without_the_calls_module(elsewhere, monkeypatch):
    """The module needs torch's and Python's headers; a program that uses the C ABI or the GDN-2 calls does not need it."""
    def fails():
        raise RuntimeError("no headers")

    monkeypatch.setattr(gbuild, "_call_stale", lambda: True)
    monkeypatch.setattr(gbuild, "_build_call", fails)
    with pytest.raises(RuntimeError, match="no headers"):
        gbuild.build()
    assert os.path.exists(gbuild.LIB)


@pytest.mark.parametrize("what", ["torch", "python"])
def test_calls_module_of_another_torch_or_python_is_not_used(monkeypatch, what):
    """It is compiled against the internals of one of each."""
    gbuild.build()
    assert not gbuild._call_stale()
    if what == "torch":
        monkeypatch.setattr(torch, "__version__", "0.1.2")
    else:
        names = dict(sysconfig.get_config_vars(), SOABI="cpython-31-other")
        monkeypatch.setattr(sysconfig, "get_config_var", names.get)
    assert gbuild._call_stale()
    monkeypatch.setattr(attn, "_bound", None)
    with pytest.raises(RuntimeError, match="not built"):
        attn.load()
