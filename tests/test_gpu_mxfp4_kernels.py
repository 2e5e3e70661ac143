"""Each kernel of the microscaled 4-bit products, forced, at the sizes where
its tiles, stages and row groups begin and end (needs an MI355X)."""
import numpy as np
import pytest

import mxfp4_reference as R
import precision_integer_gemm_amd as L
from test_gpu_mxfp4 import SPLITS, dev, dtypes, guarded, held, run_grouped, torch  # noqa: F401

pytestmark = pytest.mark.gpu

TILED = {64: L.KERNEL_TILED_64, 128: L.KERNEL_TILED_128, 256: L.KERNEL_TILED_256}


@pytest.fixture
def forced():
    """Forces a kernel for the test's calls."""
    yield L.lpgemm_set_kernel_override
    L.lpgemm_set_kernel_override(L.KERNEL_AUTO)


# rows around every tile height, columns around every width, K of one to many stages, odd unit counts
SIZES = [(1, 1, 1), (3, 5, 129), (31, 65, 256), (33, 63, 257), (64, 64, 640), (65, 129, 700), (128, 127, 896), (129, 257, 1024), (191, 96, 1152),
         (193, 256, 2000), (255, 513, 384), (256, 300, 128), (257, 8, 2560), (300, 1000, 513), (520, 260, 3200)]


@pytest.mark.parametrize("kind", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("tile", list(TILED))
@pytest.mark.parametrize("M,N,K", SIZES)
def test_tiled_product(torch, forced, kind, tile, M, N, K):  # noqa: F811
    rng = np.random.default_rng(M + N + K)
    a, sa = R.random_operand(rng, M, K)
    b, sb = R.random_operand(rng, N, K, center=117)
    out, ok = guarded(torch, (M, N), dtypes(torch)[kind])
    forced(TILED[tile])
    L.lpgemm_mxfp4(*dev(torch, a, sa, b, sb), out=out)
    assert ok()
    held(out, R.values(a, sa), R.values(b, sb), kind)


@pytest.mark.parametrize("tile", list(TILED))
def test_tiled_many_tiles_per_workgroup(torch, forced, tile):  # noqa: F811
    """More tiles than workgroups, of several heights: a workgroup goes from one to the next."""
    M, N, K = {64: (1100, 2500, 384), 128: (2000, 4200, 300), 256: (1300, 17000, 200)}[tile]
    rng = np.random.default_rng(tile)
    a, sa = R.random_operand(rng, M, K)
    b, sb = R.random_operand(rng, N, K)
    t = dev(torch, a, sa, b, sb)
    forced(TILED[tile])
    for kind in ("bfloat16", "float32"):
        held(L.lpgemm_mxfp4(*t, dtype=dtypes(torch)[kind]), R.values(a, sa), R.values(b, sb), kind)


@pytest.mark.parametrize("tile", list(TILED))
@pytest.mark.parametrize("split", list(SPLITS))
@pytest.mark.parametrize("N,K", [(96, 512), (301, 2897), (600, 40)])
def test_tiled_grouped(torch, forced, tile, split, N, K):  # noqa: F811
    forced(TILED[tile])
    run_grouped(torch, np.random.default_rng(N), SPLITS[split], N, K, "bfloat16")


@pytest.mark.parametrize("tile", list(TILED))
@pytest.mark.parametrize("split", ["single rows", "empty ones", "skewed", "tile edges", "many"])
def test_tiled_grouped_gathered_rows(torch, forced, tile, split):  # noqa: F811
    rng = np.random.default_rng(9)
    rows = rng.integers(0, 50, int(np.sum(SPLITS[split])))
    rows[::7], rows[3::11], rows[5::13], rows[6::17] = -1, 50, 2 ** 31 - 1, -2 ** 31
    forced(TILED[tile])
    out = run_grouped(torch, rng, SPLITS[split], 200, 700, "float32", T=50, rows=rows)
    assert not out[::7].any()


@pytest.mark.parametrize("tile", list(TILED))
def test_tiled_many_groups(torch, forced, tile):  # noqa: F811
    """The most groups there may be, most of them of a few rows: tile numbers past one wave's scan."""
    rng = np.random.default_rng(11)
    sizes = rng.choice([0, 0, 1, 2, 5], L.MXFP4_MAX_GROUPS)
    sizes[700] = 300
    forced(TILED[tile])
    run_grouped(torch, rng, list(sizes), 40, 140, "float32")


# ---- the narrow kernel ----------------------------------------------------------
# K around each number of waves that split it (4, 8, 16 units) and of stages a wave holds; strips that end past N
NARROW = [(1, 1, 1), (2, 15, 100), (16, 16, 512), (17, 17, 513), (32, 33, 640), (5, 100, 1024), (9, 250, 1025), (31, 48, 2048), (16, 4000, 2049),
          (3, 300, 4096), (33, 40, 700), (65, 130, 4000), (100, 100, 16384), (1000, 64, 2000), (32, 5000, 4097), (16, 100, 8192), (20, 31, 8193), (1, 9000, 300), (32, 500, 16384), (7, 4, 16300), (12, 70000, 384)]


@pytest.mark.parametrize("kind", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("M,N,K", NARROW)
def test_narrow_product(torch, forced, kind, M, N, K):  # noqa: F811
    rng = np.random.default_rng(M + N + K)
    a, sa = R.random_operand(rng, M, K)
    b, sb = R.random_operand(rng, N, K, center=117)
    out, ok = guarded(torch, (M, N), dtypes(torch)[kind])
    forced(L.KERNEL_SKINNY)
    L.lpgemm_mxfp4(*dev(torch, a, sa, b, sb), out=out)
    assert ok()
    held(out, R.values(a, sa), R.values(b, sb), kind)


@pytest.mark.parametrize("split", list(SPLITS))
@pytest.mark.parametrize("N,K", [(96, 512), (301, 2897), (600, 40), (40, 9000), (17, 1100)])
def test_narrow_grouped(torch, forced, split, N, K):  # noqa: F811
    if np.sum(SPLITS[split]) > 896:
        pytest.skip("more rows than the narrow kernel takes")
    forced(L.KERNEL_SKINNY)
    run_grouped(torch, np.random.default_rng(N), SPLITS[split], N, K, "bfloat16")


@pytest.mark.parametrize("split", ["single rows", "empty ones", "skewed", "many", "one large"])
def test_narrow_grouped_gathered_rows(torch, forced, split):  # noqa: F811
    rng = np.random.default_rng(9)
    rows = rng.integers(0, 50, int(np.sum(SPLITS[split])))
    rows[::7], rows[3::11], rows[5::13], rows[6::17] = -1, 50, 2 ** 31 - 1, -2 ** 31
    forced(L.KERNEL_SKINNY)
    out = run_grouped(torch, rng, SPLITS[split], 200, 700, "float32", T=50, rows=rows)
    assert not out[::7].any()


def test_narrow_many_groups(torch, forced):  # noqa: F811
    rng = np.random.default_rng(11)
    sizes = rng.choice([0, 0, 0, 1, 2], 512)
    sizes[300] = 60
    forced(L.KERNEL_SKINNY)
    run_grouped(torch, rng, list(sizes), 40, 140, "float32")


def test_narrow_refuses_what_it_does_not_serve(torch, forced):  # noqa: F811
    forced(L.KERNEL_SKINNY)
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    for M, U in ((4097, 4), (4, 129)):
        with pytest.raises(L.LpgemmError):
            L.lpgemm_mxfp4(z(M, 64 * U), z(M, 4 * U), z(8, 64 * U), z(8, 4 * U))
