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


def test_binding_of_another_pytorch(monkeypatch):
    # a module that says it was compiled against another version, or that says nothing, is not called
    torch = pytest.importorskip("torch")
    import types

    import sum_check_prover_b200 as fp
    for version, taken in ((str(torch.__version__), True), ("1.0", False)):
        module = types.SimpleNamespace(torch=version)
        monkeypatch.setitem(sys.modules, "sum_check_prover_b200._binding", module)
        monkeypatch.setattr(fp, "_binding", module, raising=False)
        monkeypatch.setattr(fp, "_bound", None)
        assert fp._load_binding() is (module if taken else fp._Unbound)


def test_binding_is_this_interpreters_and_pytorchs():
    torch = pytest.importorskip("torch")
    import sysconfig

    import sum_check_prover_b200 as fp
    build.build()
    assert build.BINDING.name == "_binding" + sysconfig.get_config_var("EXT_SUFFIX")
    assert not (build.HERE / "_binding.so").exists()
    if build.BINDING.exists():
        got = fp._load_binding()
        assert got is not fp._Unbound and got.torch == str(torch.__version__)


def test_binding_is_built_again_for_another_pytorch(monkeypatch, tmp_path):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(build, "BINDING", tmp_path / "_binding.so")
    monkeypatch.setattr(build, "OBJ", tmp_path / "obj")
    monkeypatch.setenv("CXX", "false")  # (a build would fail and say so)
    (tmp_path / "obj").mkdir()
    (tmp_path / "_binding.so").write_bytes(b"")
    stamp = tmp_path / "obj" / "_binding.so.torch"
    stamp.write_text(str(torch.__version__))
    assert build.build_binding() == build.BINDING
    stamp.write_text("1.0")
    with pytest.warns(UserWarning, match="was not built"):
        assert build.build_binding() is None
