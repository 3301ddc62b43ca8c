"""The build beside the library: the compiled binding of the layer operators, which may be missing."""

import sys

import pytest

from sum_check_prover_b200 import build


@pytest.mark.parametrize("compiler", ["false", "/nowhere/to/be/found", "true"])
def test_library_without_a_binding(monkeypatch, tmp_path, compiler):
    # a compiler that fails, is missing or writes nothing: a warning, no older module left, and the library as it was
    pytest.importorskip("torch")
    older = tmp_path / "_binding.so"
    older.write_bytes(b"built for another library")
    monkeypatch.setattr(build, "BINDING", older)
    monkeypatch.setenv("CXX", compiler)
    with pytest.warns(UserWarning, match="was not built"):
        assert build.build_binding(force=True) is None
    assert list(tmp_path.iterdir()) == []
    assert build.LIB.exists()


def test_binding_without_pytorch(monkeypatch, tmp_path):
    older = tmp_path / "_binding.so"
    older.write_bytes(b"built for a PyTorch that has gone")
    monkeypatch.setattr(build, "BINDING", older)
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build.build_binding() is None and not older.exists()


def test_methods_without_a_binding(monkeypatch):
    import sum_check_prover_b200 as fp
    monkeypatch.setattr(fp, "_bound", None)
    monkeypatch.setitem(sys.modules, "sum_check_prover_b200._binding", None)  # its import fails
    monkeypatch.delattr(fp, "_binding", raising=False)
    assert fp._load_binding() is fp._Unbound
    assert fp._bound.matmul_i8(1, 2) is None
