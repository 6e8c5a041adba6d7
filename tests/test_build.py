"""The build: the library stands on its own, whatever becomes of the module that
takes PyTorch tensors to it.  (Compilers are stand-ins.)"""
import os
import sys

import pytest

from exact_attention_forward_04_gb300 import _build


@pytest.fixture
def out(tmp_path, monkeypatch):
    """An empty output folder and a quick stand-in for the library's compilers."""
    monkeypatch.setattr(_build, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(_build, "LIB_PATH", str(tmp_path / "libfa_fwd.so"))
    monkeypatch.setattr(_build, "TORCH_PATH", str(tmp_path / "fa_torch.so"))
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(f"#!{sys.executable}\nimport sys\nopen(sys.argv[sys.argv.index('-o') + 1], 'w').write('built')\n")
    nvcc.chmod(0o755)
    monkeypatch.setattr(_build, "_nvcc", lambda: str(nvcc))
    return tmp_path


def compiler(code, status):
    """A command in the place of g++: writes its output file, then ends with ``status``."""
    return lambda path: [sys.executable, "-c", f"open({path!r}, 'w').write({code!r}); raise SystemExit({status})"]


def names(out):
    return sorted(n for n in os.listdir(out) if n != "nvcc")


def test_both(out, monkeypatch):
    monkeypatch.setattr(_build, "_torch_command", compiler("module", 0))
    assert _build.needs_build()
    assert _build.build() == str(out / "libfa_fwd.so")
    assert {"fa_torch.so", "libfa_fwd.so", "ptxas_report.txt"} <= set(names(out))
    assert not _build.needs_build()


def test_a_module_that_does_not_compile(out, monkeypatch):
    monkeypatch.setattr(_build, "_torch_command", compiler("half", 1))
    with pytest.warns(UserWarning, match="fa_torch"):
        assert _build.build() == str(out / "libfa_fwd.so")
    assert names(out) == ["libfa_fwd.so", "ptxas_report.txt"]


def test_no_compiler_for_the_module(out, monkeypatch):
    monkeypatch.setattr(_build, "_torch_command", lambda path: ["/nonexistent/g++", path])
    with pytest.warns(UserWarning, match="fa_torch"):
        _build.build()
    assert names(out) == ["libfa_fwd.so", "ptxas_report.txt"]

    def no_torch(path):
        raise ImportError("no PyTorch")

    monkeypatch.setattr(_build, "_torch_command", no_torch)
    with pytest.warns(UserWarning, match="no PyTorch"):
        _build.build(force=True)


def test_a_library_that_does_not_compile(out, monkeypatch):
    """An error, and no temporary file of either stays."""
    monkeypatch.setattr(_build, "_torch_command", compiler("module", 0))
    (out / "nvcc").write_text(f"#!{sys.executable}\nraise SystemExit(1)\n")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        _build.build()
    assert "libfa_fwd.so" not in names(out) and not [n for n in names(out) if ".tmp" in n or n.endswith(".o")]
