"""The torch binding belongs to one torch and one Python: built for others it is built again,
and not loaded."""

import pytest

import __graft_entry__
import paged_kv_cache_345_b200 as pa

build = __graft_entry__._build_module()


@pytest.fixture
def current(monkeypatch, tmp_path):
    """A build that is up to date by its files, whatever the files here are."""
    source, lib, binding, stamp = (tmp_path / n for n in ("pa_torch.cpp", "libpa.so", "_pa_torch.so", "stamp"))
    for p in (source, lib, binding):
        p.write_text("")
    stamp.write_text(build.built_for())
    monkeypatch.setattr(build, "LIB", str(lib))
    monkeypatch.setattr(build, "BINDING_LIB", str(binding))
    monkeypatch.setattr(build, "STAMP", str(stamp))
    monkeypatch.setattr(build, "_inputs", lambda: [])
    monkeypatch.setattr(build, "BINDING", str(source))
    return stamp


def test_files_and_versions_as_built(current):
    assert build.up_to_date()


def test_another_torch_or_python_makes_it_stale(current, monkeypatch):
    real = build.built_for()
    assert "torch" in real
    monkeypatch.setattr(build.importlib.metadata, "version", lambda name: "0.0.1")
    assert build.built_for() != real and not build.up_to_date()
    monkeypatch.undo()


def test_no_record_of_what_it_was_built_for_makes_it_stale(current):
    current.unlink()
    assert not build.up_to_date()


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch):
    torch = pytest.importorskip("torch")
    assert pa._native().built_for.split()[0] == torch.__version__
    monkeypatch.setattr(pa, "_native_module", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(ImportError, match="0.0.1"):
        pa._native()
    monkeypatch.undo()
    assert pa._native() is not None
