"""The steps of the Python build: the HIP libraries need hipcc alone, so the
codec builds where g++ or torch's headers do not fit the module over the layer
library, which fails in its own step, loudly."""
import subprocess

import pytest

from dequantize_reduce_transfer_amd import build


def test_the_libraries_build_without_a_host_compiler(monkeypatch, tmp_path):
    commands = []

    def run(cmd, **kwargs):
        commands.append(cmd)
        if cmd[0] != build.HIPCC:
            return subprocess.CompletedProcess(cmd, 1, "", "no such compiler")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    for name in ("BUILD_DIR", "LIB_PATH", "LAYER_LIB_PATH", "BINDING_PATH"):
        monkeypatch.setattr(build, name, str(tmp_path / name))
    assert build.build() == build.LIB_PATH
    assert (tmp_path / "LIB_PATH").exists() and (tmp_path / "LAYER_LIB_PATH").exists()
    assert len(commands) == len(build.SOURCES) + len(build.LAYER_SOURCES) + 2
    with pytest.raises(RuntimeError, match="no such compiler"):
        build.build_binding()
    assert not (tmp_path / "BINDING_PATH").exists()
