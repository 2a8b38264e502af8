"""The in-tree build, in a folder of its own; the library's objects are taken from
the real one."""
import importlib
import os
import shutil

import pytest

b = importlib.import_module("transformer_attention_tcgen05_gb300.build")


@pytest.fixture
def fresh(tmp_path, monkeypatch):
    b.build()
    real = b.OUT
    monkeypatch.setattr(b, "OUT", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libattn.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_attn_native.so"))

    def compile_(src, obj, verbose):
        shutil.copy(os.path.join(real, os.path.basename(obj)), obj)
        return ""
    monkeypatch.setattr(b, "_compile", compile_)
    compile_binding = b._compile_binding

    def binding(obj):
        if "CXX" in os.environ:
            return compile_binding(obj)
        return compile_(None, obj, False)
    monkeypatch.setattr(b, "_compile_binding", binding)
    monkeypatch.delenv("CXX", raising=False)
    return tmp_path


def test_libattn_is_built_where_the_binding_cannot_be(fresh, monkeypatch):
    b.build()
    assert os.path.exists(b.LIB) and os.path.exists(b.BINDING)
    os.remove(b.LIB)
    monkeypatch.setenv("CXX", "/bin/false")
    with pytest.warns(RuntimeWarning, match="binding was not built"):
        assert b.build(force=True) == b.LIB
    assert os.path.exists(b.LIB)
    # an older binding is not left for the new library
    assert not os.path.exists(b.BINDING)
    monkeypatch.delenv("CXX")
    b.build()
    assert os.path.exists(b.BINDING)


@pytest.mark.parametrize("other", ["torch", "python"])
def test_the_binding_is_built_again_for_another_torch_or_python(fresh, monkeypatch, other):
    import sysconfig

    import torch
    b.build()
    at = os.path.getmtime(b.BINDING), os.path.getmtime(b.LIB)
    b.build()
    assert at == (os.path.getmtime(b.BINDING), os.path.getmtime(b.LIB))
    if other == "torch":
        monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    else:
        real = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "other" if n == "SOABI" else real(n))
    b.build()
    assert os.path.getmtime(b.BINDING) > at[0] and os.path.getmtime(b.LIB) == at[1]
    again = os.path.getmtime(b.BINDING)
    b.build()
    assert os.path.getmtime(b.BINDING) == again
