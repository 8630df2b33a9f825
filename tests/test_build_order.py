"""The C library is built whatever becomes of the Python binding's call."""
import os
import subprocess

import pytest

from sparse_tiled_gemm_amd import build as B


def test_the_library_needs_no_python_headers(monkeypatch, tmp_path):
    """A failing compiler of the extension module is reported, after the
    library has been linked."""
    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(B, "PYCALL", str(tmp_path / "_pycall.so"))
    monkeypatch.setattr(B, "HIPCC", "hipcc")
    monkeypatch.setenv("CC", "no-such-compiler")
    compiled = []
    monkeypatch.setattr(B, "_compile", lambda src, asm, verbose: compiled.append(src))

    def run(cmd, **kw):
        if cmd[0] == "no-such-compiler":
            raise FileNotFoundError(cmd[0])
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0)

    monkeypatch.setattr(B.subprocess, "run", run)
    with pytest.raises(FileNotFoundError):
        B.build()
    assert os.path.exists(B.LIB) and sorted(compiled) == sorted(B.SOURCES)
    assert not os.path.exists(B.PYCALL)
