"""The build gives libhca.so whatever becomes of the extension module."""
import importlib.util
import os

import pytest

from long_context_compressed_hca_b200 import build as hbuild


@pytest.fixture
def built(tmp_path, monkeypatch):
    """The build in a folder of its own, without compilers: the outputs of the commands it ran."""
    ran = []

    def out(path):
        with open(path, "w"):
            ran.append(os.path.basename(path))
    monkeypatch.setattr(hbuild, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(hbuild, "LIB", str(tmp_path / "libhca.so"))
    monkeypatch.setattr(hbuild, "CALL", str(tmp_path / "_torch_call.so"))
    monkeypatch.setattr(hbuild, "_compile", lambda src, obj, extra, verbose: out(obj) or "")
    monkeypatch.setattr(hbuild, "_compile_call", lambda obj, verbose: out(obj))
    monkeypatch.setattr(hbuild, "_run", lambda cmd, what, verbose: out(cmd[cmd.index("-o") + 1]))
    return ran


def test_a_failing_extension_leaves_the_library(built, monkeypatch):
    def fail(obj, verbose):
        raise RuntimeError("no headers of torch")
    monkeypatch.setattr(hbuild, "_compile_call", fail)
    with pytest.raises(RuntimeError, match="no headers"):
        hbuild.build()
    assert os.path.exists(hbuild.LIB) and not os.path.exists(hbuild.CALL)


def test_without_torch_there_is_no_extension(built, monkeypatch):
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, package=None: None)
    assert hbuild.build() == hbuild.LIB and os.path.exists(hbuild.LIB)
    assert not any("torch_call" in x for x in built)


def test_both_are_built_and_not_built_again(built):
    hbuild.build()
    assert os.path.exists(hbuild.LIB) and os.path.exists(hbuild.CALL)
    n = len(built)
    hbuild.build()
    assert len(built) == n
