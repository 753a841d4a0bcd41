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


def test_module_of_another_torch_is_rebuilt(monkeypatch, tmp_path):
    """A module compiled against another torch or Python fails at import, whatever the files' dates say."""
    b.build()
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write("".join(a for a in cmd if a.startswith("-D")).encode())
        return type("R", (), dict(returncode=0, stdout="", stderr=""))()
    assert b._built_for(b.OPS).decode() == f"torch {b._torch_version()} {b.sys.implementation.cache_tag}"
    monkeypatch.setattr(b.subprocess, "run", run)
    b._build_ops(False)
    assert not ran                                     # just built
    monkeypatch.setattr(b, "OPS", str(tmp_path / "_ops.so"))
    b._build_ops(False)
    assert len(ran) == 1 and os.path.exists(b.OPS)
    b._build_ops(False)
    assert len(ran) == 1
    monkeypatch.setattr(b, "_torch_version", lambda: "0.0.0")
    b._build_ops(False)
    assert len(ran) == 2
    b._build_ops(False)
    assert len(ran) == 2
