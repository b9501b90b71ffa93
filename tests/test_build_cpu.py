"""The build where the paged cache's Python module cannot be made (no g++, no Python
headers): the library is there all the same, and the error says what is not. With
stand-ins for the compilers."""
import os
import subprocess

import pytest

from bit_block_quantized_nibble_amd import build as B


@pytest.mark.parametrize("fails", ["compiler", "headers", "link"])
def test_library_is_built_without_the_call_module(tmp_path, monkeypatch, fails):
    lib, calls = str(tmp_path / "libqbn.so"), str(tmp_path / "_kvcall.so")
    monkeypatch.setattr(B, "LIB", lib)
    monkeypatch.setattr(B, "CALLS", calls)
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "objects"))

    def run(cmd, **kw):
        if cmd[0] == "g++":
            if fails == "compiler":
                raise FileNotFoundError("g++")
            if fails == "headers" or "-shared" in cmd:
                return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B.subprocess, "run", run)
    open(calls, "w").close()  # of an earlier build
    with pytest.raises(RuntimeError, match="_kvcall.so"):
        B.build()
    assert os.path.exists(lib) and not os.path.exists(calls)
