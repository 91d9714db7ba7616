"""When build() compiles anew: the Python binding goes with the torch that it was compiled against."""
import importlib.metadata

import pytest

from paged_kv_attention_25_gb300 import build as pkv_build
from paged_kv_attention_25_gb300 import pkv


def another_torch(monkeypatch):
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "9.9.9")


def test_another_torch_makes_the_binding_stale(monkeypatch):
    pkv_build.build()
    assert not pkv_build._lib_stale() and not pkv_build._binding_stale()
    another_torch(monkeypatch)
    assert pkv_build._binding_stale() and not pkv_build._lib_stale()


def test_a_binding_for_another_torch_is_not_loaded(monkeypatch):
    pkv_build.build()
    monkeypatch.setattr(pkv, "_binding", None)
    another_torch(monkeypatch)
    with pytest.raises(RuntimeError, match="another torch"):
        pkv._load_binding()
