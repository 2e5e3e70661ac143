"""The tiled microscaled products where a workgroup goes from tile to tile,
each kernel by the plan that names it (needs an MI355X).

K is four units or more, so that scales come through their ring, and there are
more tiles than workgroups, of changing heights; every element is compared."""
import numpy as np
import pytest

import mxfp4_reference as R
import precision_integer_gemm_amd as L
from test_gpu_mxfp4 import dev, dtypes, guarded, held, torch  # noqa: F401
from test_gpu_mxfp4_kernels import TILED, forced  # noqa: F401

pytestmark = pytest.mark.gpu
KINDS = ["float32", "bfloat16", "float16"]


def runs(groups, N, K, E, tile_m, tile_n):
    """A call with these groups' rows takes such tiles, and more of them than workgroups."""
    p = L.lpgemm_mxfp4_plan(int(np.sum(groups)), N, K, E)
    assert (p["kernel"], p["tile_m"], p["tile_n"], p["k_split"]) == ("tiled", tile_m, tile_n, 1), p
    assert p["workgroups"] < sum(-(-n // tile_m) for n in groups) * -(-N // tile_n), p


def product(torch, M, N, K):  # noqa: F811
    rng = np.random.default_rng(M + N + K)
    a, sa = R.random_operand(rng, M, K)
    b, sb = R.random_operand(rng, N, K, center=117)
    t, va, vb = dev(torch, a, sa, b, sb), R.values(a, sa), R.values(b, sb)
    for kind in KINDS:
        out, ok = guarded(torch, (M, N), dtypes(torch)[kind])
        L.lpgemm_mxfp4(*t, out=out)
        assert ok()
        held(out, va, vb, kind, kind)


# units of a row odd and even; heights of 64, 128, 192 and 256 rows side by side
@pytest.mark.parametrize("tile,M,N,K", [(64, 1100, 2500, 640), (64, 1100, 2500, 1100), (128, 2300, 4300, 512), (128, 2200, 4300, 1153),
                                        (256, 1300, 17000, 512), (256, 1300, 12000, 1100), (256, 700, 24000, 641), (256, 66, 70000, 900)])
def test_forced(torch, forced, tile, M, N, K):  # noqa: F811
    forced(TILED[tile])
    runs([M], N, K, 0, tile, tile)
    product(torch, M, N, K)


@pytest.mark.parametrize("tile_m,tile_n,M,N,K", [(64, 128, 1000, 4200, 640), (64, 128, 700, 6500, 640), (128, 128, 2600, 3300, 640), (256, 256, 6000, 5200, 640)])
def test_auto(torch, tile_m, tile_n, M, N, K):  # noqa: F811
    runs([M], N, K, 0, tile_m, tile_n)
    product(torch, M, N, K)


def grouped(torch, sizes, N, K, T):  # noqa: F811
    rng = np.random.default_rng(N + K)
    E, n = len(sizes), int(np.sum(sizes))
    a, sa = R.random_operand(rng, T or n, K)
    b, sb = R.random_operand(rng, E * N, K, center=117)
    b, sb = b.reshape(E, N, -1), sb.reshape(E, N, -1)
    offsets = np.concatenate(([0], np.cumsum(sizes))).astype(np.int32)
    rows = None
    if T:
        rows = rng.integers(0, T, n)
        rows[::17], rows[3::29] = -1, T
    t = dev(torch, a, sa, b, sb, offsets)
    trows = dev(torch, rows.astype(np.int32))[0] if T else None
    x = R.values(a, sa)
    if T:
        x = np.where(((rows >= 0) & (rows < T))[:, None], x[rows.clip(0, T - 1)], 0.0)
    for kind in KINDS:
        out, ok = guarded(torch, (n, N), dtypes(torch)[kind])
        L.lpgemm_mxfp4_grouped(*t, rows=trows, out=out)
        assert ok()
        for e in range(E):
            i, j = offsets[e], offsets[e + 1]
            if j > i:
                held(out[i:j], x[i:j], R.values(b[e], sb[e]), kind, f"group {e} {kind}")


MIXED = [64, 130, 0, 192, 256, 300, 1, 65, 513, 700, 0, 128, 257, 63, 450]
MANY = [[5, 64, 0, 129, 200, 256, 30, 1, 90, 0][i % 10] for i in range(80)]


@pytest.mark.parametrize("T", [0, 400])
@pytest.mark.parametrize("tile", list(TILED))
@pytest.mark.parametrize("sizes,N,K", [(MIXED, 6000, 640), (MIXED, 5900, 1100), (MANY, 1500, 513)])
def test_forced_grouped(torch, forced, tile, sizes, N, K, T):  # noqa: F811
    forced(TILED[tile])
    runs(sizes, N, K, len(sizes), tile, tile)
    grouped(torch, sizes, N, K, T)


@pytest.mark.parametrize("T", [0, 400])
@pytest.mark.parametrize("tile_m,tile_n,E,each,N,K", [(64, 128, 64, 9, 1100, 640), (128, 128, 20, 65, 3300, 640), (256, 256, 80, 130, 2100, 640)])
def test_auto_grouped(torch, tile_m, tile_n, E, each, N, K, T):  # noqa: F811
    runs([each] * E, N, K, E, tile_m, tile_n)
    grouped(torch, [each] * E, N, K, T)
