"""The library is built without what only its Python binding needs (nvcc, no GPU)."""
import os
import sys
import warnings

import pytest

from paged_kv_cache_301_gb300 import build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A library of one function, with a binding that does not compile."""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (csrc / "binding.cpp").write_text("#error no such header\n")
    for name, path in (("CSRC", csrc), ("BUILD", tmp_path / "build"),
                       ("LIB", tmp_path / "lib.so"), ("BINDING", tmp_path / "binding.so"),
                       ("BINDING_SOURCE", csrc / "binding.cpp"), ("PKG", tmp_path),
                       ("STAMP", tmp_path / "build" / "machine.txt"),
                       ("BINDING_STAMP", tmp_path / "build" / "binding.txt")):
        monkeypatch.setattr(build, name, str(path), raising=False)
    monkeypatch.setattr(build, "SOURCES", ["one.cu"])
    monkeypatch.setattr(build, "HEADERS", [])
    return tmp_path


@pytest.mark.parametrize("without", ["headers", "torch"])
def test_library_without_a_binding(small, monkeypatch, without):
    if without == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)        # import torch fails
    (small / "binding.so").write_text("of another Python")
    with pytest.warns(RuntimeWarning, match="binding"):
        lib = build.build()
    assert os.path.exists(lib) and (small / "build" / "machine.txt").exists()
    assert not (small / "binding.so").exists()
    made = os.path.getmtime(lib)
    with pytest.warns(RuntimeWarning, match="binding"):
        build.build()
    assert os.path.getmtime(lib) == made                       # not built again
    with pytest.raises((RuntimeError, ImportError)):
        build.build(need_binding=True)


def test_a_binding_is_built_once(small):
    (small / "csrc" / "binding.cpp").write_text("int two() { return 2; }\n")
    real = build._link_binding
    links = []
    build._link_binding = lambda obj: (links.append(obj), (small / "binding.so").write_text("x"))
    try:
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            build.build()
            build.build(need_binding=True)
    finally:
        build._link_binding = real
    assert len(links) == 1


def test_a_missing_binding_is_named(monkeypatch):
    import paged_kv_cache_301_gb300 as pa
    build.build()
    monkeypatch.setattr(pa, "_native", None)
    monkeypatch.setitem(sys.modules, "paged_kv_cache_301_gb300._binding", None)
    monkeypatch.delattr(pa, "_binding", raising=False)
    with pytest.raises(ImportError, match="_binding.so"):
        pa.pa_rope_append(*[None] * 9)
    pa.lib()                                                   # the others do not need it
