"""When the compiled part of the binding is built anew."""
import os

import __graft_entry__
from exact_attention_blackwell_tiled_gb300 import _build

HEADER = os.path.join(_build.INCLUDE, "fa.h")


def test_binding_is_linked_to_this_torch(monkeypatch, tmp_path):
    __graft_entry__.build()
    assert not _build._binding_stale(HEADER)
    # another torch in the same tree
    (tmp_path / "version.py").write_text("__version__ = '0.0.0'\n")
    with monkeypatch.context() as m:
        m.setattr(_build, "_torch_dir", lambda: str(tmp_path))
        assert _build._binding_stale(HEADER)
    with monkeypatch.context() as m:  # a binary of before the key was written
        m.setattr(_build, "BINDING_KEY_PATH", _build.BINDING_KEY_PATH + ".missing")
        assert _build._binding_stale(HEADER)
    assert not _build._binding_stale(HEADER)
