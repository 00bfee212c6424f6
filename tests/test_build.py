"""The library's build where a part of it cannot be made."""
import ctypes

import pytest

from contextual_sparsity_sparse_gb300 import build as cb


def test_the_library_is_linked_without_pythons_headers(tmp_path, monkeypatch):
    """The cache calls' module needs Python.h; what needs only the library must not go with it.  The failure is still told."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(cb, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(cb, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(cb, "QCALL", str(tmp_path / "qcall.so"))
    monkeypatch.setattr(cb, "sources", lambda: [str(src)])
    monkeypatch.setattr(cb.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "nowhere")})
    with pytest.raises(RuntimeError, match="qcall.c"):
        cb.build(force=True)
    assert ctypes.CDLL(str(tmp_path / "lib.so")).one() == 1
    assert not (tmp_path / "qcall.so").exists()
