"""What build() makes of the installed torch: the C library needs none.  (Nothing of the package itself is rebuilt here:
the module's path, its compiler's command and torch's place are stand-ins.)"""
import importlib.util
import os
import types

import pytest

from paged_kv_attention_gqa_gb300 import build as B


@pytest.fixture
def made(monkeypatch, tmp_path):
    """Counts how often the module is compiled, into a folder of its own."""
    B.build()
    count = []
    monkeypatch.setattr(B, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(B, "_marshal_command", lambda out: count.append(out) or ["touch", out])
    return count


def without_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_the_library_is_built_without_torch(monkeypatch, tmp_path, capfd):
    B.build()
    monkeypatch.setattr(B, "MARSHAL", str(tmp_path / "_marshal.so"))
    without_torch(monkeypatch)
    monkeypatch.setattr(B, "OUT", str(tmp_path / "libpkv.so"))
    assert B.build() == B.OUT and os.path.exists(B.OUT)
    assert not os.path.exists(B.MARSHAL)
    text = capfd.readouterr().err
    assert "torch" in text and "speculative" in text, text


def test_the_library_is_built_where_the_module_does_not_compile(made, monkeypatch, tmp_path):
    monkeypatch.setattr(B, "_marshal_command", lambda out: ["false"])
    monkeypatch.setattr(B, "OUT", str(tmp_path / "libpkv.so"))
    with pytest.raises(RuntimeError, match="marshal.cpp"):
        B.build()
    assert os.path.exists(B.OUT) and not os.path.exists(B.MARSHAL)


def test_the_module_follows_torch(made, monkeypatch, tmp_path):
    """It is compiled against torch's headers: another torch, in another place or in the same, takes another module."""
    B.build()
    B.build()
    assert len(made) == 1 and os.path.exists(B.MARSHAL)
    folder = tmp_path / "torch"
    folder.mkdir()
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: types.SimpleNamespace(origin=str(folder / "__init__.py")) if name == "torch" else find(name, *a))
    for i, version in enumerate(("1.0", "1.0", "1.1", "1.1")):
        (folder / "version.py").write_text(f"__version__ = '{version}'\n")
        B.build()
        assert len(made) == 2 + i // 2, (i, version)
