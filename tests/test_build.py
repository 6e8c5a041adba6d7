"""The build: the library stands on its own, whatever becomes of the module that
takes PyTorch tensors to it.  (Compilers are stand-ins.)"""
import importlib
import os
import sys

import pytest
import torch

import exact_attention_forward_04_gb300 as fa
from exact_attention_forward_04_gb300 import _build

ROPE, CACHE = (importlib.import_module(f"exact_attention_forward_04_gb300.{m}") for m in ("rope", "cache_e2m1"))


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


def test_a_module_of_another_pytorch_is_stale(out, monkeypatch):
    monkeypatch.setattr(_build, "_torch_command", compiler("module", 0))
    _build.build()
    library = (out / "libfa_fwd.so").stat().st_mtime_ns
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert _build.needs_build()
    _build.build()
    assert not _build.needs_build() and "0.0.1" in _build.torch_built_for()
    assert (out / "libfa_fwd.so").stat().st_mtime_ns == library     # the library is not


@pytest.mark.parametrize("content,note", ((None, None), ("not a library", True), ("not a library", None),
                                          ("not a library", "another PyTorch")))
def test_a_module_that_does_not_load(out, monkeypatch, content, note):
    """The calls then go through Python, which refuses here, as there is no GPU's tensor."""
    monkeypatch.setattr(fa, "load_library", lambda: None)
    if content:
        (out / "fa_torch.so").write_text(content)
    if note:
        (out / "fa_torch.txt").write_text(_build.torch_key() if note is True else note)
    with pytest.warns(RuntimeWarning, match="through Python"):
        m = fa._load_torch()
    assert m.rope(1, 2, 3, False, False) is None and m.read(1, 1.0, 1.0, 2) is None
    assert not m.append(*range(9)) and m.forward(*range(11)) is None
    monkeypatch.setattr(ROPE, "_usual", m.rope)
    monkeypatch.setattr(CACHE, "_usual", m)
    x, pos = torch.zeros(4, 2, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fa.rope(x, pos, fa.rope_table(16, 32, device="cpu"))
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache_read_e2m1(fa.CacheE2M1(torch.zeros(2, 2, 1, 18 * 64, dtype=torch.uint8)), pos.long())


@pytest.mark.gpu
def test_calls_without_the_module(monkeypatch):
    """The same bits as with it."""
    g = torch.Generator().manual_seed(1)
    k, v, q = (torch.randn(40, h, 64, generator=g).to(torch.bfloat16).cuda() for h in (2, 2, 6))
    table, pos = fa.rope_table(64, 64), torch.arange(40, dtype=torch.int32, device="cuda")
    blocks, lens, cu = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([[2, 0, 1]], [40], [0, 40]))
    slots = blocks[0, pos.long() // 16].long() * 16 + pos % 16

    def step():
        cache = fa.cache_alloc_e2m1(3, 2, 16, 64, 0.25, 0.5)
        fa.cache_append_e2m1(k, v, cache, slots, positions=pos, table=table)
        x = fa.rope(q, pos, table)
        return [cache.data, x, fa.rope_backward(q, pos, table), *fa.cache_read_e2m1(cache, slots),
                *fa.cache_forward_e2m1(x, cache, blocks, lens, cu)]

    with_it = step()
    monkeypatch.setattr(_build, "TORCH_PATH", "/nonexistent/fa_torch.so")
    monkeypatch.setattr(ROPE, "_usual", None)
    monkeypatch.setattr(CACHE, "_usual", None)
    with pytest.warns(RuntimeWarning, match="through Python"):
        without = step()
    fa.check_errors()
    assert all(torch.equal(a, b) for a, b in zip(with_it, without))
