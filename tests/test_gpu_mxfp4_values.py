"""Every k, every place of a scale and every scale byte through each kernel of
the microscaled products (needs an MI355X)."""
import numpy as np
import pytest

import mxfp4_reference as R
import precision_integer_gemm_amd as L
from test_gpu_mxfp4 import dev, dtypes, held, torch  # noqa: F401
from test_gpu_mxfp4_kernels import forced  # noqa: F401

pytestmark = pytest.mark.gpu

KERNELS = {"64": L.KERNEL_TILED_64, "128": L.KERNEL_TILED_128, "256": L.KERNEL_TILED_256, "narrow": L.KERNEL_SKINNY}


def one_k_each(rows, K, first=0):
    """Row i holds 1.5 (code 3, scale 1) at k = first + i and zeros."""
    codes = np.zeros((rows, 64 * R.units(K)), np.uint8)
    k = first + np.arange(rows)
    codes[np.arange(rows), k // 2] = 3 << 4 * (k % 2)
    return codes, np.full((rows, 4 * R.units(K)), 127, np.uint8)


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("K", [300, 1100, 2049])
def test_every_k(torch, forced, kernel, K):  # noqa: F811
    b, sb = R.random_operand(np.random.default_rng(K), 70, K)
    a, sa = one_k_each(K, K)
    t = dev(torch, a, sa, b, sb)
    want = 1.5 * R.values(b, sb)[:, :K].T
    forced(KERNELS[kernel])
    np.testing.assert_array_equal(L.lpgemm_mxfp4(*t, dtype=torch.float32).cpu().numpy(), want)


@pytest.mark.parametrize("M,K", [(1, 500), (16, 1100), (16, 8200), (32, 8200), (16, 16384)])
def test_every_k_few_rows(torch, forced, M, K):  # noqa: F811
    """Each number of stages that the narrow kernel's waves hold."""
    b, sb = R.random_operand(np.random.default_rng(K), 40, K)
    vb = R.values(b, sb)
    tb = dev(torch, b, sb)
    forced(L.KERNEL_SKINNY)
    got = []
    for first in range(0, K - M + 1, M):
        got.append(L.lpgemm_mxfp4(*dev(torch, *one_k_each(M, K, first)), *tb, dtype=torch.float32))
    got = torch.cat(got).cpu().numpy()
    np.testing.assert_array_equal(got, 1.5 * vb[:, :len(got)].T)
    assert K - len(got) < M  # the last ones, too
    last = L.lpgemm_mxfp4(*dev(torch, *one_k_each(M, K, K - M)), *tb, dtype=torch.float32).cpu().numpy()
    np.testing.assert_array_equal(last, 1.5 * vb[:, K - M:K].T)


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("K", [300, 1100, 2049])
def test_every_k_grouped(torch, forced, kernel, K):  # noqa: F811
    """Groups of 0 to 40 rows, gathered: row i of the result is a k of its own."""
    rng = np.random.default_rng(K)
    a, sa = one_k_each(K, K)
    ta = dev(torch, a, sa)
    forced(KERNELS[kernel])
    for first in range(0, K, 800):
        order = first + rng.permutation(min(800, K - first))
        cuts = np.minimum(np.cumsum(np.r_[0, rng.integers(0, 41, 60)]), len(order))
        cuts[-1] = len(order)
        E = len(cuts) - 1
        b, sb = R.random_operand(rng, E * 40, K)
        b, sb = b.reshape(E, 40, -1), sb.reshape(E, 40, -1)
        got = L.lpgemm_mxfp4_grouped(*ta, *dev(torch, b, sb, cuts.astype(np.int32)), rows=dev(torch, order.astype(np.int32))[0],
                                     dtype=torch.float32).cpu().numpy()
        for e in range(E):
            i = slice(cuts[e], cuts[e + 1])
            np.testing.assert_array_equal(got[i], 1.5 * R.values(b[e], sb[e])[:, order[i]].T)


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("K", [128, 300, 1100, 4000])
def test_every_scale_byte(torch, forced, kernel, K):  # noqa: F811
    """Bytes of 0 to 254 in A's blocks against 254 to 0 in B's: products of scales near 1, each far from its row's others."""
    M, N, blocks = 45, 90, -(-K // 32)
    forced(KERNELS[kernel])
    for kind in ("float32", "bfloat16"):
        for seed in range(3):
            rng = np.random.default_rng(seed)
            a, sa = R.random_operand(rng, M, K)
            b, sb = R.random_operand(rng, N, K)
            center = rng.integers(0, 255, blocks)
            center[rng.permutation(blocks)[:2]] = 0, 254
            sa[:, :blocks] = np.clip(center + rng.integers(-4, 5, (M, blocks)), 0, 254)
            sb[:, :blocks] = np.clip(254 - center + rng.integers(-4, 5, (N, blocks)), 0, 254)
            got = L.lpgemm_mxfp4(*dev(torch, a, sa, b, sb), dtype=dtypes(torch)[kind])
            held(got, R.values(a, sa), R.values(b, sb), kind, f"seed {seed}")


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("K", [90, 300, 500, 1100, 2049])
def test_nan_scale_in_every_block(torch, forced, kernel, K):  # noqa: F811
    """Row i of A (column i of B) has its NaN in block i; the last one has none."""
    blocks = -(-K // 32)
    rng = np.random.default_rng(K)
    a, sa = R.random_operand(rng, blocks + 1, K)
    b, sb = R.random_operand(rng, blocks + 1, K)
    i = np.arange(blocks)
    forced(KERNELS[kernel])
    bad = sa.copy()
    bad[i, i] = 255
    got = L.lpgemm_mxfp4(*dev(torch, a, bad, b, sb)).float().cpu().numpy()
    assert np.isnan(got[:-1]).all() and np.isfinite(got[-1]).all()
    bad = sb.copy()
    bad[i, i] = 255
    got = L.lpgemm_mxfp4(*dev(torch, a, sa, b, bad)).float().cpu().numpy()
    assert np.isnan(got[:, :-1]).all() and np.isfinite(got[:, -1]).all()
