"""The microscaled product's workspace argument: checked and passed on, and
nothing is sized or allocated for it, as no kernel takes scratch memory."""
import pytest
import torch

import precision_integer_gemm_amd as L
from precision_integer_gemm_amd import _binding


@pytest.fixture
def launched(monkeypatch):
    """The long way up to the library, with operands on the host; the launch's arguments."""
    _binding._mx_torch()
    seen = []
    monkeypatch.setattr(_binding, "_mx_units", lambda codes, scales, name, dim, device=None: codes.shape[-1] // 64)
    monkeypatch.setattr(_binding, "_mx_out", lambda out, dtype, M, N, device: (out, L.OUT_BF16))
    monkeypatch.setattr(_binding, "_mx_launch", lambda function, index, stream, *args: seen.append(args))

    def none(*args):
        raise AssertionError("asked for a workspace's size")
    monkeypatch.setattr(_binding, "lpgemm_mxfp4_workspace_size", none)
    return seen


@pytest.mark.parametrize("workspace", ["auto", None])
def test_none_is_made(launched, workspace):
    a, sa = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    out = torch.zeros(4, 4, dtype=torch.bfloat16)
    assert L.lpgemm_mxfp4(a, sa, a, sa, out=out, workspace=workspace) is out
    assert launched[0][-2:] == (None, 0)


def test_its_size_is_zero():
    for sizes in ((1, 1, 1), (8192, 8192, 8192), (4, 5, 1 << 20)):
        assert L.lpgemm_mxfp4_workspace_size(*sizes) == 0
