"""What build() compiles when: the library without torch, the module on torch
tensors again for another torch (commands are recorded, not run)."""
import os
import subprocess

import pytest

from weight_only_quantized_qmoe_gb300 import build as B


class Recorder:
    """Stands in for the compilers: writes the output a command names."""

    def __init__(self):
        self.outputs = []

    def run(self, cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write("built")
        self.outputs.append(os.path.basename(out).replace(".tmp", ""))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def take(self):
        got, self.outputs = self.outputs, []
        return got


@pytest.fixture
def compilers(tmp_path, monkeypatch):
    r = Recorder()
    monkeypatch.setattr(B.subprocess, "run", r.run)
    monkeypatch.setattr(B, "nvcc_path", lambda: "/cuda/bin/nvcc")
    monkeypatch.setattr(B, "ROOT", str(tmp_path))
    monkeypatch.setattr(B, "LIB_PATH", str(tmp_path / "libqmoe.so"))
    monkeypatch.setattr(B, "TORCH_MODULE", str(tmp_path / "_ops_torch.so"))
    return r


def test_the_library_needs_no_torch(compilers, monkeypatch):
    monkeypatch.setattr(B, "find_spec", lambda name: None)
    assert B.build() == B.LIB_PATH and os.path.exists(B.LIB_PATH)
    got = compilers.take()
    assert "libqmoe.so" in got and "qmoe_api.o" in got and not any("torch" in n for n in got)
    B.build()                       # and is current without it
    assert compilers.take() == []
