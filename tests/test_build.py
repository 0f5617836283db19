"""When the library and the binding are compiled, and in which order (no GPU, no compiler)."""
import os

import pytest

from gated_delta_rule_88_b200 import build as kbuild


@pytest.fixture
def files(tmp_path, monkeypatch):
    """A library and a binding that are up to date, in a folder of their own."""
    lib, ext = tmp_path / "lib.so", tmp_path / "ext.so"
    lib.write_bytes(b"library")
    ext.write_bytes(b"\x7fELF..\0" + kbuild._built_for().encode() + b"\0..")
    monkeypatch.setattr(kbuild, "LIB", str(lib))
    monkeypatch.setattr(kbuild, "EXT", str(ext))
    monkeypatch.setattr(kbuild, "BUILD", str(tmp_path / "objects"))
    return lib, ext


class Compiler:
    """Stands in for subprocess.run: writes the output file of a command whose
    program is not among the missing ones."""

    def __init__(self, missing=()):
        self.missing, self.programs = missing, []

    def __call__(self, cmd, **kw):
        name = os.path.basename(cmd[0])
        self.programs.append(name)
        if name in self.missing:
            raise FileNotFoundError(cmd[0])
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write(b"made")
        return type("Done", (), {"returncode": 0, "stdout": "", "stderr": ""})


def test_nothing_is_compiled_again(files, monkeypatch):
    run = Compiler()
    monkeypatch.setattr(kbuild.subprocess, "run", run)
    assert not kbuild.needs_build() and not kbuild.needs_binding()
    kbuild.build()
    assert run.programs == []


def test_library_is_built_without_the_bindings_compiler(files, monkeypatch):
    """nvcc alone makes the library; that the binding is missing is still an error."""
    lib, ext = files
    lib.unlink()
    ext.unlink()
    run = Compiler(missing=("g++",))
    monkeypatch.setattr(kbuild.subprocess, "run", run)
    with pytest.raises(FileNotFoundError):
        kbuild.build()
    assert lib.read_bytes() == b"made" and set(run.programs[:-1]) == {"nvcc"} and run.programs[-1] == "g++"


@pytest.mark.parametrize("what", ["torch", "python"])
def test_binding_is_built_again_for_another_torch_or_python(files, monkeypatch, what):
    import torch

    if what == "torch":
        monkeypatch.setattr(torch, "__version__", torch.__version__ + "1")
    else:
        monkeypatch.setattr(kbuild.sys, "implementation", type("I", (), {"cache_tag": "cpython-399"}))
    run = Compiler()
    monkeypatch.setattr(kbuild.subprocess, "run", run)
    kbuild.build()
    assert run.programs == ["g++"]


def test_the_module_says_what_it_was_built_for():
    kbuild.build()
    from gated_delta_rule_88_b200 import _paged
    assert _paged.built_for == kbuild._built_for()
    assert not kbuild.needs_binding()
