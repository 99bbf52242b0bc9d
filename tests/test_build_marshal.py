"""Building the binding's tensor checks: hosts that lack what it takes, and reuse of a build."""
import sys

from speculative_decoding_tree_ddtree_gb300 import build as B


def test_the_library_is_built_without_torch(monkeypatch, capsys):
    B.build()
    monkeypatch.setitem(sys.modules, "torch", None)  # importing it fails
    assert B.build_marshal() is None and B.build_marshal(force=True) is None
    assert B.build() == B.LIB
    assert "tensor checks are not built" in capsys.readouterr().err


def test_a_build_for_another_python_is_not_loaded(monkeypatch, tmp_path):
    import shutil

    import pytest

    from speculative_decoding_tree_ddtree_gb300 import lucetree as LT
    path = B.build_marshal()
    if path is None:
        pytest.skip("the compiled check was not built here")
    monkeypatch.setattr(LT, "_PKG", str(tmp_path))
    monkeypatch.setattr(LT, "_arg", LT._arg_slow)    # as while the binding is being imported
    for name in ("_marshal.so", "_marshal.cpython-39-x86_64-linux-gnu.so", "_marshal.cpython-39-aarch64-linux-gnu.so"):
        shutil.copy(path, tmp_path / name)
    assert LT._load_marshal() is LT._arg_slow
    shutil.copy(path, tmp_path / B.os.path.basename(path))
    assert LT._load_marshal() is not LT._arg_slow


def test_a_build_that_failed_is_not_tried_every_time(monkeypatch, tmp_path):
    log, cxx = tmp_path / "log", tmp_path / "cxx"
    cxx.write_text(f"#!/bin/sh\necho run >> {log}\necho no headers >&2\nexit 1\n")
    cxx.chmod(0o755)
    monkeypatch.setenv("CXX", str(cxx))
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(B, "MARSHAL", str(tmp_path / "_marshal.so"))
    runs = lambda: len(log.read_text().split())  # noqa: E731
    assert B.build_marshal() is None and B.build_marshal() is None and runs() == 1
    assert B.build_marshal(force=True) is None and runs() == 2
    src = tmp_path / "marshal.cpp"
    src.write_text("// changed")
    monkeypatch.setattr(B, "MARSHAL_SRC", str(src))
    assert B.build_marshal() is None and runs() == 3
