"""The build without what the native half of the Python binding needs
(torch's headers, a host compiler): the library itself does not need them."""

import os

import pytest

from dequant_gemv_rht_amd import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    src, out = tmp_path / "csrc", tmp_path / "lib"
    src.mkdir()
    out.mkdir()
    (src / "a.cpp").write_text('extern "C" int answer() { return 42; }\n')
    (src / B.BINDING).write_text('#include "no_such_header.h"\n')
    monkeypatch.setattr(B, "CSRC", str(src))
    monkeypatch.setattr(B, "OUT", str(out))
    monkeypatch.setattr(B, "LIB", str(out / "libwq.so"))
    monkeypatch.setattr(B, "BINDING_LIB", str(out / "_wqpy.so"))
    return src, out


def test_library_is_built_when_the_binding_cannot_be(tree):
    _, out = tree
    (out / "_wqpy.so").write_text("of an earlier build")
    with pytest.warns(RuntimeWarning, match="no_such_header"):
        lib = B.build()
    assert os.path.exists(lib) and lib == str(out / "libwq.so")
    assert not (out / "_wqpy.so").exists()   # nothing stale in its place


def test_a_broken_library_source_still_fails(tree):
    src, out = tree
    (src / "a.cpp").write_text("int answer( {\n")
    with pytest.raises(RuntimeError, match="hipcc failed"):
        B.build()
    assert not (out / "libwq.so").exists()


def test_binding_as_it_is_compiles(tree, monkeypatch):
    _, out = tree
    monkeypatch.setattr(B, "CSRC", os.path.join(B.HERE, "csrc"))
    assert os.path.exists(B.build_binding())
