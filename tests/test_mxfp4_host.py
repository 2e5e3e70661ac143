"""Refusals of the microscaled 4-bit entry points: rejected on the host, before
any HIP call (no GPU needed)."""
import ctypes

import pytest
import torch

import precision_integer_gemm_amd as L

P = 4096  # a fake, aligned device address, never dereferenced here
QUANTIZE = dict(x=P, dtype=L.OUT_BF16, ldx=200, codes=P, scales=P, rows=4, K=200)
DEQUANTIZE = dict(codes=P, scales=P, y=P, dtype=L.OUT_BF16, rows=4, K=200)
PRODUCT = dict(a=P, sa=P, b=P, sb=P, d=P, dtype=L.OUT_BF16, M=4, N=8, K=200, ws=None, wsb=0)
GROUPED = dict(a=P, sa=P, T=4, rows=P, b=P, sb=P, E=3, offsets=P, d=P, dtype=L.OUT_BF16, R=4, N=8, K=200)
BAD, UNS = L.ERR_INVALID_ARG, L.ERR_UNSUPPORTED

CASES = [
    *[("lpgemm_mxfp4_quantize", QUANTIZE, c, w) for c, w in [
        ({"rows": -1}, BAD), ({"K": -1}, BAD), ({"dtype": L.OUT_FP8_E4M3}, BAD), ({"dtype": 9}, BAD), ({"x": None}, BAD),
        ({"codes": None}, BAD), ({"scales": None}, BAD), ({"x": P + 1}, BAD), ({"codes": P + 8}, BAD), ({"scales": P + 2}, BAD),
        ({"ldx": 199}, BAD), ({"ldx": -200}, BAD), ({"rows": 4, "ldx": 2 ** 61}, BAD), ({"K": L.MXFP4_MAX_K + 1, "ldx": 1 << 21}, UNS),
        ({"rows": 2 ** 60}, UNS), ({"dtype": L.OUT_F32, "x": P + 2}, BAD)]],
    *[("lpgemm_mxfp4_dequantize", DEQUANTIZE, c, w) for c, w in [
        ({"rows": -1}, BAD), ({"K": -1}, BAD), ({"dtype": L.OUT_FP8_E5M2}, BAD), ({"y": None}, BAD), ({"codes": None}, BAD),
        ({"scales": None}, BAD), ({"y": P + 1}, BAD), ({"K": L.MXFP4_MAX_K + 1}, UNS)]],
    *[("lpgemm_mxfp4", PRODUCT, c, w) for c, w in [
        ({"M": -1}, BAD), ({"N": -1}, BAD), ({"K": -1}, BAD), ({"dtype": L.OUT_FP8_E4M3}, BAD), ({"d": None}, BAD), ({"a": None}, BAD),
        ({"sa": None}, BAD), ({"b": None}, BAD), ({"sb": None}, BAD), ({"d": P + 8}, BAD), ({"a": P + 8}, BAD), ({"b": P + 4}, BAD),
        ({"sa": P + 1}, BAD), ({"sb": P + 2}, BAD), ({"K": L.MXFP4_MAX_K + 1}, UNS), ({"M": 2 ** 31}, UNS), ({"N": 2 ** 31}, UNS),
        ({"ws": None, "wsb": 256}, BAD), ({"ws": P + 16, "wsb": 256}, BAD)]],
    *[("lpgemm_mxfp4_grouped", GROUPED, c, w) for c, w in [
        ({"T": -1}, BAD), ({"R": -1}, BAD), ({"N": -1}, BAD), ({"K": -1}, BAD), ({"E": -1}, BAD), ({"dtype": 7}, BAD), ({"d": None}, BAD),
        ({"a": None}, BAD), ({"b": None}, BAD), ({"offsets": None}, BAD), ({"offsets": P + 2}, BAD), ({"rows": P + 2}, BAD),
        ({"rows": None, "T": 5}, BAD), ({"E": L.MXFP4_MAX_GROUPS + 1}, UNS), ({"T": 2 ** 25, "K": 200}, UNS), ({"sb": P + 1}, BAD)]],
]


@pytest.mark.parametrize("fn,args,change,want", CASES, ids=[f"{c[0][7:]}-{c[2]}" for c in CASES])
def test_argument_errors(fn, args, change, want):
    assert getattr(L.lib(), fn)(*{**args, **change}.values(), None) == want


@pytest.mark.parametrize("fn,args,change", [
    ("lpgemm_mxfp4_quantize", QUANTIZE, {"rows": 0}), ("lpgemm_mxfp4_quantize", QUANTIZE, {"K": 0, "x": None, "codes": None, "scales": None}),
    ("lpgemm_mxfp4_dequantize", DEQUANTIZE, {"rows": 0, "y": None}), ("lpgemm_mxfp4", PRODUCT, {"M": 0, "a": None}),
    ("lpgemm_mxfp4", PRODUCT, {"N": 0, "b": None, "d": None}), ("lpgemm_mxfp4_grouped", GROUPED, {"R": 0, "rows": P}),
    ("lpgemm_mxfp4_grouped", GROUPED, {"E": 0, "b": None, "sb": None, "offsets": None})])
def test_nothing_to_do(fn, args, change):
    assert getattr(L.lib(), fn)(*{**args, **change}.values(), None) == L.OK


def test_workspace_size_refusals():
    n = ctypes.c_size_t(1)
    f = L.lib().lpgemm_mxfp4_workspace_size
    assert f(4, 8, 200, 0, None) == BAD
    for bad in ((-1, 8, 200), (4, -1, 200), (4, 8, -1)):
        assert f(*bad, 0, ctypes.byref(n)) == BAD
    assert f(4, 8, L.MXFP4_MAX_K + 1, 0, ctypes.byref(n)) == UNS
    for empty in ((0, 8, 200), (4, 0, 200), (4, 8, 0)):
        assert f(*empty, 0, ctypes.byref(n)) == L.OK and n.value == 0


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


class TestTensorCalls:
    """Types, shapes and devices are checked before anything is launched."""

    def test_quantize(self):
        with pytest.raises(TypeError):
            L.lpgemm_mxfp4_quantize([1.0])
        with pytest.raises(TypeError):
            L.lpgemm_mxfp4_quantize(torch.zeros(2, 32, dtype=torch.float64))
        with pytest.raises(ValueError, match="2-D"):
            L.lpgemm_mxfp4_quantize(torch.zeros(32))
        with pytest.raises(ValueError, match="GPU"):
            L.lpgemm_mxfp4_quantize(torch.zeros(2, 32))

    def test_operands(self):
        a, sa, b, sb = u8(2, 64), u8(2, 4), u8(3, 64), u8(3, 4)
        for bad in (TypeError, (a.int(), sa, b, sb)), (ValueError, (a[0], sa, b, sb)), (ValueError, (a, sa, b, sb)):
            with pytest.raises(bad[0]):
                L.lpgemm_mxfp4(*bad[1])
        with pytest.raises((TypeError, ValueError)):
            L.lpgemm_mxfp4_grouped(a, sa, b, sb, torch.zeros(4, dtype=torch.int32))
        with pytest.raises((TypeError, ValueError)):
            L.lpgemm_mxfp4_dequantize(a, sa, 128)
