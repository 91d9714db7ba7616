"""What build() makes and when: the C library needs nvcc alone, the Python binding the torch that it was compiled against."""
import importlib.metadata
import os

import pytest

from paged_kv_attention_25_gb300 import build as pkv_build
from paged_kv_attention_25_gb300 import pkv


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build of two small sources into a folder of its own."""
    for name, file in (("LIB", "libpkv.so"), ("BINDING", "pkv_binding.so"), ("BINDING_STAMP", "pkv_binding.stamp")):
        monkeypatch.setattr(pkv_build, name, str(tmp_path / file))
    monkeypatch.setattr(pkv_build, "BUILD", str(tmp_path))
    monkeypatch.setattr(pkv_build, "SOURCES", ["plan.cpp", "cache.cpp"])
    return tmp_path


def another_torch(monkeypatch):
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "9.9.9")


def test_without_torch_the_library_is_built(elsewhere, monkeypatch):
    monkeypatch.setattr(pkv_build, "_torch", lambda: None)
    assert os.path.exists(pkv_build.build())
    assert not os.path.exists(pkv_build.BINDING)
    made = os.path.getmtime(pkv_build.LIB)
    pkv_build.build()                                       # nothing is left to do
    assert os.path.getmtime(pkv_build.LIB) == made and not pkv_build._binding_stale()


def test_a_binding_that_does_not_compile_leaves_the_library(elsewhere, monkeypatch):
    broken = elsewhere / "broken.cpp"
    broken.write_text("#error no")
    monkeypatch.setattr(pkv_build, "BINDING_SOURCE", str(broken))
    with pytest.raises(RuntimeError, match="C library is built"):
        pkv_build.build()
    assert os.path.exists(pkv_build.LIB) and pkv_build._binding_stale()


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
