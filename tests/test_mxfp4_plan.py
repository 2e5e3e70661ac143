"""What lpgemm_mxfp4_plan says a microscaled product would run (host only)."""
import ctypes

import pytest

import precision_integer_gemm_amd as L
from precision_integer_gemm_amd._binding import PlanInfo


@pytest.fixture
def forced():
    yield L.lpgemm_set_kernel_override
    L.lpgemm_set_kernel_override(L.KERNEL_AUTO)


def shape(*sizes):
    p = L.lpgemm_mxfp4_plan(*sizes)
    return p["kernel"], p["tile_m"], p["tile_n"], p["k_split"]


def test_argument_errors():
    f, info = L.lib().lpgemm_mxfp4_plan, ctypes.byref(PlanInfo())
    assert f(4, 8, 200, 0, 0, None) == L.ERR_INVALID_ARG
    for bad in ((-1, 8, 200, 0), (4, -1, 200, 0), (4, 8, -1, 0), (4, 8, 200, -1)):
        assert f(*bad, 0, info) == L.ERR_INVALID_ARG
    for big in ((4, 8, L.MXFP4_MAX_K + 1, 0), (2 ** 31, 8, 200, 0), (4, 2 ** 31, 200, 0), (4, 8, 200, L.MXFP4_MAX_GROUPS + 1)):
        assert f(*big, 0, info) == L.ERR_UNSUPPORTED
    for empty in ((0, 8, 200), (4, 0, 200)):
        assert L.lpgemm_mxfp4_plan(*empty)["workgroups"] == 0


@pytest.mark.parametrize("sizes,want", [
    ((1, 4096, 4096), ("skinny", 16, 16, 8)), ((16, 28672, 8192), ("skinny", 16, 16, 4)), ((32, 500, 16384), ("skinny", 32, 16, 8)),
    ((1000, 64, 16384), ("skinny", 32, 16, 8)), ((64, 4096, 4096, 32), ("skinny", 16, 16, 1)), ((333, 1001, 2897), ("tiled", 64, 64, 1)),
    ((1024, 1024, 4096), ("tiled", 64, 64, 2)), ((1000, 4200, 640), ("tiled", 64, 128, 1)), ((4096, 2048, 4096, 64), ("tiled", 64, 128, 1)),
    ((2600, 3300, 640), ("tiled", 128, 128, 1)), ((6000, 5200, 640), ("tiled", 256, 256, 1)), ((8192, 8192, 8192), ("tiled", 256, 256, 1)),
    ((13000, 1100, 640, 100), ("tiled", 256, 256, 1)), ((16384, 4096, 4096, 32), ("tiled", 256, 256, 1)), ((50, 8192, 16500), ("tiled", 64, 64, 2))])
def test_what_auto_picks(sizes, want):
    assert shape(*sizes) == want


def test_forced_kernels(forced):
    for kernel, tile in ((L.KERNEL_TILED_64, 64), (L.KERNEL_TILED_128, 128), (L.KERNEL_TILED_256, 256)):
        forced(kernel)
        assert shape(3000, 3000, 512)[:3] == shape(300, 40, 2000, 7)[:3] == ("tiled", tile, tile)
    for K in (0, 1, 200, 384):  # rows of fewer than four units
        assert shape(3000, 3000, K)[:3] == ("tiled", 128, 128)
    assert shape(3000, 3000, 385)[:3] == ("tiled", 256, 256)
    forced(L.KERNEL_SKINNY)
    assert shape(4096, 100, 16384)[0] == shape(896, 100, 40000, 512)[0] == "skinny"
    for refused in ((4097, 100, 200), (4, 100, 16385), (897, 100, 200, 5), (10, 100, 200, 513)):
        with pytest.raises(L.LpgemmError):
            L.lpgemm_mxfp4_plan(*refused)
    forced(L.KERNEL_FP6)
    with pytest.raises(L.LpgemmError):
        L.lpgemm_mxfp4_plan(300, 300, 512)


def test_workgroups():
    for cu in (1, 8, 256, 304):
        for sizes in ((6000, 5200, 640), (333, 1001, 2897), (64, 4096, 4096, 32), (4096, 2048, 4096, 64), (1, 28672, 512), (4096, 64, 16384)):
            p = L.lpgemm_mxfp4_plan(*sizes, **({} if len(sizes) == 4 else {"E": 0}), cu_count=cu)
            assert 1 <= p["workgroups"] <= (2 * cu if p["kernel"] == "tiled" else max(cu, -(-sizes[0] // p["tile_m"])))
            assert p["threads"] in (256, 512)
