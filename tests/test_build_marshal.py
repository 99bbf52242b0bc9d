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
