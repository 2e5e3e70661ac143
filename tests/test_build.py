"""What the build needs: the C library and the probe want hipcc alone, the
Python module of the tensor calls also PyTorch, Python's headers and g++."""
import os
import shutil
import sys

import pytest
import torch

import precision_integer_gemm_amd as L
from precision_integer_gemm_amd import _binding, build


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """build() into a folder of its own, every command only recorded."""
    for name in ("LIB", "CALLS_LIB", "PROBE_LIB"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    seen = []

    def run(cmd, what, verbose):
        seen.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(build, "run", run)
    monkeypatch.setattr(build, "hipcc", lambda: "/opt/rocm/bin/hipcc")
    return seen


def made(folder):
    return sorted(os.listdir(folder))


def test_everything(commands, tmp_path):
    if shutil.which("g++") is None or torch.version.hip is None:
        pytest.skip("needs g++ and PyTorch for ROCm")
    build.build()
    assert made(tmp_path) == ["_ceiling.so", "_lpgemm.so", "_tensor_calls.so"]


@pytest.mark.parametrize("without", ["torch", "g++", "Python.h"])
def test_the_library_needs_hipcc_alone(commands, monkeypatch, tmp_path, without, capsys):
    if without == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    elif without == "g++":
        which = shutil.which
        monkeypatch.setattr(shutil, "which", lambda n, *a, **k: None if n == "g++" else which(n, *a, **k))
    else:
        exists = os.path.exists
        monkeypatch.setattr(os.path, "exists", lambda p: False if str(p).endswith("Python.h") else exists(p))
    (tmp_path / "_tensor_calls.so").write_text("built against another library")
    build.build()
    assert made(tmp_path) == ["_ceiling.so", "_lpgemm.so"]
    assert len(commands) == 4 and all(c[0].endswith("hipcc") for c in commands)
    assert "_tensor_calls.so is not built" in capsys.readouterr().out


def test_tensor_calls_without_their_module(monkeypatch, tmp_path):
    """The checks still say what is wrong."""
    monkeypatch.setattr(_binding, "_mx", None)
    monkeypatch.setattr(_binding, "CALLS_PATH", str(tmp_path / "none.so"))
    with pytest.raises(ValueError, match="GPU"):
        L.lpgemm_mxfp4_quantize(torch.zeros(2, 32))
    assert _binding._mx[3] is _binding._LongWay
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    for call in (lambda: L.lpgemm_mxfp4_dequantize(u8(2, 64), u8(2, 4), 128), lambda: L.lpgemm_mxfp4(u8(2, 64), u8(2, 4), u8(2, 64), u8(2, 4)),
                 lambda: L.lpgemm_mxfp4_grouped(u8(2, 64), u8(2, 4), u8(1, 2, 64), u8(1, 2, 4), torch.zeros(2, dtype=torch.int32))):
        with pytest.raises(ValueError, match="GPU"):
            call()
