"""The build of the descriptor module where its tools are missing (CPU only)."""
import pytest
import torch.utils.cpp_extension

from mamba_ssd_scan_05_amd import build


@pytest.fixture
def target(tmp_path, monkeypatch):
    at = tmp_path / "_pydesc.so"
    at.write_bytes(b"of an earlier build")
    monkeypatch.setattr(build, "PYDESC", str(at))
    return at


def test_no_compiler(target, monkeypatch, capsys):
    monkeypatch.setenv("CXX", "no-such-compiler")
    assert build._compile_pydesc() is False
    assert not target.exists() and "no-such-compiler" in capsys.readouterr().err


def test_no_torch_headers(target, monkeypatch, capsys):
    monkeypatch.setattr(torch.utils.cpp_extension, "include_paths", lambda *a, **k: [])
    assert build._compile_pydesc() is False
    assert not target.exists() and "torch" in capsys.readouterr().err


def test_no_python_headers(target, monkeypatch, capsys):
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda *a, **k: {"include": "/no/such/place"})
    assert build._compile_pydesc() is False
    assert not target.exists() and "Python.h" in capsys.readouterr().err


def test_an_error_in_the_source_is_an_error(target, monkeypatch, tmp_path):
    (tmp_path / "ssd_pydesc.cpp").write_text("#error broken\n")
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    with pytest.raises(RuntimeError, match="ssd_pydesc"):
        build._compile_pydesc()
    assert target.exists()
