"""Building without what only the compiled marshalling needs: the library is built all the same."""
import os

import pytest

from partial_activation_sync_caat_b200 import build as B

FAKE = """#!/bin/sh
while [ $# -gt 0 ]; do
  if [ "$1" = -o ]; then shift; echo "%s" > "$1"; fi
  shift
done
exit %d
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Outputs in a folder of their own, compilers that only write their output."""
    def compiler(name, code=0):
        path = tmp_path / name
        path.write_text(FAKE % (name, code))
        path.chmod(0o755)
        return str(path)

    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(B, "nvcc_path", lambda: compiler("bin-nvcc"))
    monkeypatch.setattr(B, "marshal_path", lambda version=None: str(tmp_path / "marshal.so"))
    monkeypatch.setenv("CXX", compiler("cxx"))
    compiler.path = tmp_path
    return compiler


def test_both_are_built(tree):
    assert B.build() == str(tree.path / "lib.so") and (tree.path / "marshal.so").read_text() == "cxx\n"
    assert B.up_to_date() and B.marshal_up_to_date()
    os.remove(tree.path / "marshal.so")
    before = os.path.getmtime(tree.path / "lib.so")
    assert not B.marshal_up_to_date()
    B.build()
    assert B.marshal_up_to_date() and os.path.getmtime(tree.path / "lib.so") == before


@pytest.mark.parametrize("how", ["fails", "missing", "no torch"])
def test_without_the_marshalling(tree, monkeypatch, capfd, how):
    (tree.path / "marshal.so").write_text("old")
    os.utime(tree.path / "marshal.so", (0, 0))
    if how == "no torch":
        monkeypatch.setattr(B.importlib.util, "find_spec", lambda name: None)
    else:
        monkeypatch.setenv("CXX", tree("cxx", 1) if how == "fails" else str(tree.path / "none"))
    for force in (False, True):
        assert B.build(force=force) == str(tree.path / "lib.so")
        assert B.up_to_date()
    # what another version of the sources left is not loaded with the new library
    assert how == "no torch" or not (tree.path / "marshal.so").exists()
    err = capfd.readouterr().err
    assert ("marshal" in err and "cxx" in err or "none" in err) == (how != "no torch")
    assert "nvcc" not in err


def test_a_library_that_does_not_compile_is_an_error(tree, monkeypatch):
    monkeypatch.setattr(B, "nvcc_path", lambda: tree("bad-nvcc", 1))
    with pytest.raises(RuntimeError, match="nvcc failed"):
        B.build()
    assert not B.up_to_date()


def test_without_nvcc_a_current_library_is_enough(tree, monkeypatch):
    B.build()

    def none():
        raise RuntimeError("nvcc not found")

    monkeypatch.setattr(B, "nvcc_path", none)
    os.remove(tree.path / "marshal.so")
    assert B.build() == str(tree.path / "lib.so")
    with pytest.raises(RuntimeError):
        B.build(force=True)
