"""What build() does when the marshalling module cannot be built or belongs to another torch."""
import os

import pytest

from conformer_speech_recognition_b200 import build as b


def test_library_is_linked_when_the_module_fails(monkeypatch, tmp_path):
    """The C ABI needs nvcc alone: a compiler error of the Python module is reported after the library is there."""
    b.build()
    lib = tmp_path / "libgam.so"
    monkeypatch.setattr(b, "LIB", str(lib))

    def fail(force):
        raise RuntimeError("g++ failed")
    monkeypatch.setattr(b, "_build_ops", fail)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        b.build()
    assert lib.exists() and lib.stat().st_size > 1 << 20


def test_library_is_built_without_torch(monkeypatch, tmp_path):
    b.build()
    lib = tmp_path / "libgam.so"
    monkeypatch.setattr(b, "LIB", str(lib))
    monkeypatch.setattr(b, "OPS", str(tmp_path / "_ops.so"))
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None)
    b.build()
    assert lib.exists() and not os.path.exists(b.OPS)
