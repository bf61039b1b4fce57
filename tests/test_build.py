"""The build: what it leaves where the torch binding cannot be compiled, and when a
binding that is there is not the one that is wanted."""
import os

import pytest

from exact_attention_51_gb300 import build as eabuild


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The built objects, linked into another folder."""
    eabuild.build()
    monkeypatch.setattr(eabuild, "_compile", lambda src, extra=(): (
        os.path.join(eabuild.BUILD_DIR, os.path.basename(src) + ".o"), ""))
    monkeypatch.setattr(eabuild, "LIB_PATH", str(tmp_path / eabuild.LIB_NAME))
    monkeypatch.setattr(eabuild, "BINDING_PATH", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(eabuild, "STAMP_PATH", str(tmp_path / "binding.stamp"))
    return tmp_path


def test_the_library_is_linked_where_the_binding_does_not_compile(elsewhere, monkeypatch):
    def fails():
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(eabuild, "_compile_binding", fails)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        eabuild.build(force=True)
    assert sorted(os.listdir(elsewhere)) == [eabuild.LIB_NAME]
    assert not eabuild.up_to_date()


def test_without_torch_the_library_alone_is_built(elsewhere, monkeypatch):
    found = eabuild.importlib.util.find_spec
    monkeypatch.setattr(eabuild.importlib.util, "find_spec", lambda name: None if name == "torch" else found(name))
    assert eabuild.build() == eabuild.LIB_PATH
    assert sorted(os.listdir(elsewhere)) == [eabuild.LIB_NAME]
    assert eabuild.up_to_date()


def test_a_binding_of_another_torch_or_python_is_made_again(monkeypatch, tmp_path):
    eabuild.build()
    assert eabuild.up_to_date()
    stamp = eabuild._read_stamp()
    version = eabuild.importlib.metadata.version
    with monkeypatch.context() as m:
        m.setattr(eabuild.importlib.metadata, "version", lambda name: "2.0.0" if name == "torch" else version(name))
        assert not eabuild.up_to_date()
    with monkeypatch.context() as m:
        m.setattr(eabuild.sysconfig, "get_config_var", lambda name: "cpython-399-other")
        assert not eabuild.up_to_date()
    with monkeypatch.context() as m:
        m.setattr(eabuild, "STAMP_PATH", str(tmp_path / "none"))  # a binding that no build has finished
        assert not eabuild.up_to_date()
    assert eabuild.up_to_date() and eabuild._read_stamp() == stamp
