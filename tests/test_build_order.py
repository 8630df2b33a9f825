"""The C library is built whatever becomes of the Python binding's call."""
import os
import subprocess
import sys

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


def test_a_missing_extension_module_is_named():
    """As a missing library: what to run."""
    code = ("import sys; sys.modules['sparse_tiled_gemm_amd._pycall'] = None\n"
            "from sparse_tiled_gemm_amd import gemm as G\n"
            "try:\n"
            "    G.gemm_q8_store(0, 0, 'bf16', None, 0, None, None, stream=0)\n"
            "except RuntimeError as e:\n"
            "    assert 'sparse_tiled_gemm_amd.build' in str(e), e\n"
            "else:\n"
            "    raise AssertionError\n")
    subprocess.run([sys.executable, "-c", code], check=True, cwd=B.ROOT)
