"""What a built native binding belongs to: the header and the source that it was compiled from, and the library."""
import os
import shutil

import pytest

from packed_variable_length_varlen_gb300 import build


@pytest.fixture(scope="module")
def va():
    build.build()
    build.binding()
    from packed_variable_length_varlen_gb300 import varlen_attn
    return varlen_attn


@pytest.fixture
def apart(va, monkeypatch, tmp_path):
    """The binding and the library with what says where they come from, in a folder of their own."""
    for name, path in (("BINDING", build.BINDING), ("LIB", build.LIB)):
        for f in os.listdir(build.BUILD):
            if f.startswith(os.path.basename(path)):
                shutil.copy(os.path.join(build.BUILD, f), tmp_path)
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(path)))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    return tmp_path


class _Lib:
    def __init__(self, name):
        self._name = name


def _loads(va):
    """Whether a process with this folder would take the binding (it is not loaded a second time here)."""
    return build.binding_built(build.LIB)


def test_as_built(va, apart):
    assert _loads(va)


@pytest.mark.parametrize("which", ["HEADER", "BINDING_SOURCE"])
def test_another_header_or_source(va, apart, monkeypatch, which):
    other = apart / "other"
    with open(getattr(build, which)) as f:
        other.write_text(f.read() + "\n// more\n")
    monkeypatch.setattr(build, which, str(other))
    assert not _loads(va)
    assert va._load_binding(_Lib(build.LIB)) is None


def test_a_header_that_is_not_there(va, apart, monkeypatch):
    monkeypatch.setattr(build, "HEADER", str(apart / "missing"))
    assert not _loads(va)
    assert va._load_binding(_Lib(build.LIB)) is None


def test_a_library_of_another_header(va, apart):
    for text in ("another", None):
        if text is None:
            os.remove(build.LIB + ".header")
        else:
            (apart / (os.path.basename(build.LIB) + ".header")).write_text(text)
        assert not _loads(va)
        assert va._load_binding(_Lib(build.LIB)) is None
        assert not build.up_to_date(build.LIB)


def test_a_build_that_fails_leaves_no_binding(va, apart, monkeypatch):
    """The module of the build before is not taken for one of this source."""
    monkeypatch.setenv("CXX", "/bin/false")
    with pytest.raises(RuntimeError):
        build.binding(force=True)
    assert not _loads(va)
    assert va._load_binding(_Lib(build.LIB)) is None


def test_an_entry_that_fails_to_build_goes_by_ctypes(va, apart, monkeypatch, capsys):
    """build() of the repository's entry points goes on without the binding, and no stale one is left to load."""
    import __graft_entry__ as entry
    monkeypatch.setenv("CXX", "/bin/false")
    monkeypatch.setattr(build, "build", lambda *a, **k: build.LIB)
    os.utime(build.BINDING, (0, 0))
    (apart / (os.path.basename(build.BINDING) + ".tag")).write_text("another")
    entry.build()
    assert "no native binding" in capsys.readouterr().err
    assert not _loads(va)
