"""Refusals and plans of the block-scaled e4m3 entry points: rejected on the host,
before any HIP call (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_block_reference as R
import precision_integer_gemm_amd as L
from precision_integer_gemm_amd._binding import PlanInfo

P = 4096  # a fake, aligned device address, never dereferenced here
QUANTIZE = dict(x=P, dtype=L.OUT_BF16, ldx=200, block_rows=1, pow2=0, codes=P, scales=P, rows=4, K=200)
DEQUANTIZE = dict(codes=P, scales=P, block_rows=128, y=P, dtype=L.OUT_BF16, rows=4, K=200)
PRODUCT = dict(a=P, sa=P, b=P, sb=P, block_rows=128, d=P, dtype=L.OUT_BF16, M=4, N=8, K=200)
GROUPED = dict(a=P, sa=P, T=4, rows=P, b=P, sb=P, block_rows=1, E=3, offsets=P, d=P, dtype=L.OUT_BF16, R=4, N=8, K=200)
BAD, UNS = L.ERR_INVALID_ARG, L.ERR_UNSUPPORTED

CASES = [
    *[("lpgemm_fp8_block_quantize", QUANTIZE, c, w) for c, w in [
        ({"rows": -1}, BAD), ({"K": -1}, BAD), ({"dtype": L.OUT_FP8_E4M3}, BAD), ({"dtype": 9}, BAD), ({"x": None}, BAD), ({"codes": None}, BAD),
        ({"scales": None}, BAD), ({"x": P + 1}, BAD), ({"codes": P + 8}, BAD), ({"scales": P + 2}, BAD), ({"ldx": 199}, BAD), ({"ldx": -200}, BAD),
        ({"block_rows": 0}, BAD), ({"block_rows": 64}, BAD), ({"block_rows": -128}, BAD), ({"pow2": 2}, BAD), ({"pow2": -1}, BAD),
        ({"ldx": 2 ** 61}, BAD), ({"K": L.FP8_BLOCK_MAX_K + 1, "ldx": 1 << 21}, UNS), ({"rows": 2 ** 60}, UNS), ({"dtype": L.OUT_F32, "x": P + 2}, BAD)]],
    *[("lpgemm_fp8_block_dequantize", DEQUANTIZE, c, w) for c, w in [
        ({"rows": -1}, BAD), ({"K": -1}, BAD), ({"dtype": L.OUT_FP8_E5M2}, BAD), ({"y": None}, BAD), ({"codes": None}, BAD), ({"scales": None}, BAD),
        ({"block_rows": 2}, BAD), ({"y": P + 1}, BAD), ({"K": L.FP8_BLOCK_MAX_K + 1}, UNS)]],
    *[("lpgemm_fp8_block", PRODUCT, c, w) for c, w in [
        ({"M": -1}, BAD), ({"N": -1}, BAD), ({"K": -1}, BAD), ({"dtype": L.OUT_FP8_E4M3}, BAD), ({"d": None}, BAD), ({"a": None}, BAD), ({"sa": None}, BAD),
        ({"b": None}, BAD), ({"sb": None}, BAD), ({"d": P + 8}, BAD), ({"a": P + 8}, BAD), ({"b": P + 4}, BAD), ({"sa": P + 1}, BAD), ({"sb": P + 2}, BAD),
        ({"block_rows": 127}, BAD), ({"K": L.FP8_BLOCK_MAX_K + 1}, UNS), ({"M": 2 ** 31}, UNS), ({"N": 2 ** 31}, UNS)]],
    *[("lpgemm_fp8_block_grouped", GROUPED, c, w) for c, w in [
        ({"T": -1}, BAD), ({"R": -1}, BAD), ({"N": -1}, BAD), ({"K": -1}, BAD), ({"E": -1}, BAD), ({"dtype": 7}, BAD), ({"d": None}, BAD), ({"a": None}, BAD),
        ({"b": None}, BAD), ({"offsets": None}, BAD), ({"offsets": P + 2}, BAD), ({"rows": P + 2}, BAD), ({"rows": None, "T": 5}, BAD),
        ({"block_rows": 3}, BAD), ({"E": L.FP8_BLOCK_MAX_GROUPS + 1}, UNS), ({"T": 2 ** 24, "K": 200}, UNS), ({"sb": P + 1}, BAD)]],
]


@pytest.mark.parametrize("fn,args,change,want", CASES, ids=[f"{c[0][7:]}-{c[2]}" for c in CASES])
def test_argument_errors(fn, args, change, want):
    assert getattr(L.lib(), fn)(*{**args, **change}.values(), None) == want


@pytest.mark.parametrize("fn,args,change", [
    ("lpgemm_fp8_block_quantize", QUANTIZE, {"rows": 0}), ("lpgemm_fp8_block_quantize", QUANTIZE, {"K": 0, "x": None, "codes": None, "scales": None}),
    ("lpgemm_fp8_block_dequantize", DEQUANTIZE, {"rows": 0, "y": None}), ("lpgemm_fp8_block", PRODUCT, {"M": 0, "a": None}),
    ("lpgemm_fp8_block", PRODUCT, {"N": 0, "b": None, "d": None}), ("lpgemm_fp8_block_grouped", GROUPED, {"R": 0}),
    ("lpgemm_fp8_block_grouped", GROUPED, {"E": 0, "b": None, "sb": None, "offsets": None})])
def test_nothing_to_do(fn, args, change):
    assert getattr(L.lib(), fn)(*{**args, **change}.values(), None) == L.OK


def test_plan_errors():
    f, info = L.lib().lpgemm_fp8_block_plan, ctypes.byref(PlanInfo())
    assert f(4, 8, 200, 0, 0, None) == BAD
    for bad in ((-1, 8, 200, 0), (4, -1, 200, 0), (4, 8, -1, 0), (4, 8, 200, -1)):
        assert f(*bad, 0, info) == BAD
    for big in ((4, 8, L.FP8_BLOCK_MAX_K + 1, 0), (2 ** 31, 8, 200, 0), (4, 2 ** 31, 200, 0), (4, 8, 200, L.FP8_BLOCK_MAX_GROUPS + 1)):
        assert f(*big, 0, info) == UNS
    for empty in ((0, 8, 200), (4, 0, 200)):
        assert L.lpgemm_fp8_block_plan(*empty)["workgroups"] == 0


@pytest.mark.parametrize("sizes,want", [
    ((1, 4096, 4096), ("skinny", 16)), ((16, 28672, 8192), ("skinny", 16)), ((16, 500, 28672), ("skinny", 16)), ((32, 4096, 4096), ("skinny", 32)),
    ((32, 28672, 8192), ("tiled", 64)), ((100, 100, 16384), ("skinny", 16)), ((64, 4096, 4096, 32), ("skinny", 16)), ((333, 1001, 2897), ("tiled", 64)),
    ((1024, 1024, 4096), ("tiled", 64)), ((1024, 4096, 4096), ("tiled", 128)), ((2848, 2880, 3200), ("tiled", 256)), ((8192, 8192, 8192), ("tiled", 256)),
    ((16384, 4096, 4096, 32), ("tiled", 256))])
def test_what_auto_picks(sizes, want):
    p = L.lpgemm_fp8_block_plan(*sizes)
    assert (p["kernel"], p["tile_m"]) == want


@pytest.mark.parametrize("kernel", [L.KERNEL_GENERAL, L.KERNEL_FP6])
def test_kernels_it_has_not(kernel):
    L.lpgemm_set_kernel_override(kernel)
    try:
        assert L.lib().lpgemm_fp8_block_plan(100, 100, 100, 0, 0, ctypes.byref(PlanInfo())) == UNS
    finally:
        L.lpgemm_set_kernel_override(L.KERNEL_AUTO)


class TestTensorCalls:
    """Types, shapes and devices are checked before anything is launched."""

    def test_quantize(self):
        q = L.lpgemm_fp8_block_quantize
        for bad, what in (([1.0], TypeError), (torch.zeros(2, 32, dtype=torch.float64), TypeError), (torch.zeros(32), ValueError)):
            with pytest.raises(what):
                q(bad)
        with pytest.raises(ValueError, match="GPU"):
            q(torch.zeros(2, 32))
        with pytest.raises(ValueError, match="block_rows"):
            q(torch.zeros(2, 32), block_rows=64)

    def test_operands(self):
        c = lambda *s: torch.zeros(s, dtype=torch.float8_e4m3fn)  # noqa: E731
        f = lambda *s: torch.zeros(s)  # noqa: E731
        for bad in ((c(2, 128).float(), f(2, 1), c(3, 128), f(3, 1)), (c(2, 128), f(2, 1).half(), c(3, 128), f(3, 1)),
                    (c(2, 128), f(2, 1), c(3, 128), f(3, 1)), (c(128), f(1), c(3, 128), f(3, 1))):
            with pytest.raises((TypeError, ValueError)):
                L.lpgemm_fp8_block(*bad)
            with pytest.raises((TypeError, ValueError)):
                L.lpgemm_fp8_block_grouped(*bad, torch.zeros(4, dtype=torch.int32))
        with pytest.raises((TypeError, ValueError)):
            L.lpgemm_fp8_block_dequantize(c(2, 128), f(2, 1), 128)


class TestReference:
    def test_values_and_codes_are_pytorch_s(self):
        codes = torch.arange(256, dtype=torch.uint8)
        want = codes.view(torch.float8_e4m3fn).float().numpy()
        np.testing.assert_array_equal(R.VALUES.astype(np.float32), want)
        x = torch.cat((torch.randn(20000) * 100, torch.randn(20000) * 0.01, torch.tensor([0.0, -0.0, 448.0, 2.0 ** -10, 3 * 2.0 ** -10]))).clamp(-448, 448)
        np.testing.assert_array_equal(R.encode(x.double().numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())

    @pytest.mark.parametrize("block_rows", [1, 128])
    @pytest.mark.parametrize("pow2", [False, True])
    def test_quantised_values_are_near(self, block_rows, pow2):
        x = np.random.default_rng(0).standard_normal((200, 300)).astype(np.float32)
        codes, scales = R.quantize(x, block_rows, pow2)
        off = np.abs(R.values(codes, scales)[:, :300] - x)
        step = np.repeat(R.by_row(scales, 200), 128, 1)[:, :300]
        # half a step: 2^-4 of a normal code's value, 2^-10 of the scale below; the inverse's rounding
        assert (off <= 1.001 * np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * step)).all()
        assert (R.VALUES[codes] <= 448).all()
        if pow2:
            assert (np.frexp(scales)[0] == 0.5).all()
