"""The build of the Python binding: what is left behind when a compilation does not end well."""
import os

import pytest

from linear_attention_06_gb300 import build as kbuild


class Compiler:
    """Stands in for the compiler's process: `code` is its exit status, None if the build is cut short in it."""
    started, code = 0, 0

    def __init__(self, cmd, **kw):
        type(self).started += 1
        self.out, self.returncode = cmd[cmd.index("-o") + 1], type(self).code

    def communicate(self):
        if self.returncode is None:
            raise KeyboardInterrupt
        if self.returncode == 0:
            with open(self.out, "w") as f:
                f.write("new")
        return b"", None


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build directory of its own, with no CUDA sources, and an older binding beside a stamp of another torch."""
    monkeypatch.setattr(kbuild, "BUILD", str(tmp_path))
    monkeypatch.setattr(kbuild, "BINDING", str(tmp_path / "_latent.so"))
    monkeypatch.setattr(kbuild, "STAMP", str(tmp_path / "latent_binding.txt"), raising=False)
    monkeypatch.setattr(kbuild, "LIB", str(tmp_path / "libkda.so"))
    monkeypatch.setattr(kbuild, "sources", lambda: [])
    monkeypatch.setattr(kbuild.subprocess, "Popen", Compiler)
    Compiler.started, Compiler.code = 0, 0
    (tmp_path / "libkda.so").write_text("library")
    (tmp_path / "_latent.so").write_text("old")
    (tmp_path / "latent_binding.txt").write_text("torch 0 python 0\n")
    return tmp_path


def test_a_compilation_cut_short_leaves_no_older_binding_that_seems_to_fit(tree):
    Compiler.code = None
    with pytest.raises(KeyboardInterrupt):
        kbuild.build()
    assert not os.path.exists(kbuild.BINDING)
    Compiler.code = 0
    kbuild.build()
    assert Compiler.started == 2 and open(kbuild.BINDING).read() == "new"


def test_a_compilation_that_fails_is_tried_again(tree):
    Compiler.code = 1
    for _ in range(2):
        with pytest.raises(RuntimeError, match="compilation failed"):
            kbuild.build()
        assert not os.path.exists(kbuild.BINDING)
    assert Compiler.started == 2


def test_a_binding_for_this_torch_is_kept(tree):
    kbuild.build()
    kbuild.build()
    assert Compiler.started == 1 and open(kbuild.BINDING).read() == "new"
