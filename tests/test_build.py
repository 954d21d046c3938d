"""What the build makes of the PyTorch it finds; nothing is compiled here."""

import sys
import types

import pytest

from memory_bound_cnn_amd import build


@pytest.fixture
def linked(monkeypatch):
    """The names of the files that a build links, with the compilers left out."""
    out = []
    monkeypatch.setattr(build, "_compile", lambda src: (src + ".o", ""))
    monkeypatch.setattr(build, "_link", lambda cmd, to: out.append(to))
    return out


@pytest.mark.parametrize("torch", [None, types.SimpleNamespace(__file__="/nowhere/torch/__init__.py",
                                                               version=types.SimpleNamespace(hip=None))])
def test_library_is_built_without_pytorch_for_these_gpus(linked, monkeypatch, capsys, torch):
    """The C library needs none; the PyTorch module is left out, and said to be."""
    monkeypatch.setitem(sys.modules, "torch", torch)
    assert build.build() == build.OUT
    assert linked == [build.OUT]
    assert "_tokens" in capsys.readouterr().err


def test_library_and_module_are_built_with_it(linked, monkeypatch):
    commands = []
    monkeypatch.setattr(build.subprocess, "run", lambda cmd, **k: commands.append(cmd) or types.SimpleNamespace(returncode=0))
    assert build.build() == build.OUT
    assert linked == [build.OUT, build.TORCH_OUT] and len(commands) == 1


def test_a_module_that_does_not_compile_is_an_error(linked, monkeypatch):
    monkeypatch.setattr(build.subprocess, "run",
                        lambda cmd, **k: types.SimpleNamespace(returncode=1, stdout="", stderr="no"))
    with pytest.raises(RuntimeError, match="wtconv_tok_torch"):
        build.build()
    assert linked == [build.OUT]
