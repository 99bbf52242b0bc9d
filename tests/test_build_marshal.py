"""Building the binding's tensor checks: hosts that lack what it takes, and reuse of a build."""
import sys

from speculative_decoding_tree_ddtree_gb300 import build as B


def test_the_library_is_built_without_torch(monkeypatch, capsys):
    B.build()
    monkeypatch.setitem(sys.modules, "torch", None)  # importing it fails
    assert B.build_marshal() is None and B.build_marshal(force=True) is None
    assert B.build() == B.LIB
    assert "tensor checks are not built" in capsys.readouterr().err
