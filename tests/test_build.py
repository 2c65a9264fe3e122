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


def test_the_module_is_built_again_for_another_torch(compilers, monkeypatch):
    monkeypatch.setattr(B, "torch_version", lambda: "2.9.1+cu130", raising=False)
    B.build()
    assert {"libqmoe.so", "_ops_torch.so"} <= set(compilers.take())
    assert B.up_to_date()
    B.build()
    assert compilers.take() == []
    monkeypatch.setattr(B, "torch_version", lambda: "2.11.0+cu130")
    assert not B.up_to_date() and B.library_up_to_date()
    B.build()
    assert compilers.take() == ["qmoe_ops_torch.o", "_ops_torch.so"]
    assert B.up_to_date()


def test_the_version_is_that_of_the_torch_there_is():
    torch = pytest.importorskip("torch")
    assert torch.__version__ in B.torch_version()
