"""The C-ABI library does not depend on what only the Python binding needs."""

import os

import pytest

from gated_deltanet_speculative_amd import build as B


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """The build with stand-ins for the compilers, into a folder of its own."""
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(B, "MARSHAL", str(tmp_path / "marshal.so"))
    monkeypatch.setattr(B, "_compile", lambda src: src + ".o")

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        if cmd[0] == "g++":
            raise FileNotFoundError("g++")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done

    monkeypatch.setattr(B.subprocess, "run", run)


def test_the_library_is_built_where_the_binding_cannot_be(fake):
    with pytest.raises(RuntimeError, match="lib.so is built.*marshal.so is not"):
        B.build(verbose=False)
    assert os.path.exists(B.LIB)


def test_the_library_alone(fake):
    assert B.build(verbose=False, binding=False) == B.LIB and os.path.exists(B.LIB)
