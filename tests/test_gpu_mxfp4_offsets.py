"""Offsets of the grouped microscaled product that fall somewhere (needs an
MI355X): an offset below one before it counts as that one, so every row has one
group at most, whatever the offsets hold."""
import numpy as np
import pytest

import mxfp4_reference as R
import precision_integer_gemm_amd as L
from test_gpu_mxfp4 import dev, guarded, held, torch  # noqa: F401
from test_gpu_mxfp4_kernels import forced  # noqa: F401

pytestmark = pytest.mark.gpu

KERNELS = {"auto": L.KERNEL_AUTO, "64": L.KERNEL_TILED_64, "128": L.KERNEL_TILED_128, "256": L.KERNEL_TILED_256, "narrow": L.KERNEL_SKINNY}
ROWS = 300


def patterns():
    rng = np.random.default_rng(6)
    up = np.linspace(0, ROWS, 201).astype(np.int64)
    dented = up.copy()
    dented[[30, 64, 65, 130, 199]] = [0, -5, ROWS, 7, 2 ** 31 - 1]
    return {"one falls": [0, 40, 20, 60, 300], "last falls": [0, 100, 200, 50], "begins high": [250, 10, 300, 280],
            "there and back": [0 if e % 2 == 0 else ROWS for e in range(41)], "there and back, many": [0 if e % 2 == 0 else ROWS for e in range(513)],
            "outside, too": [-9, 50, -2 ** 31, 2 ** 31 - 1, 0, 120], "anything": rng.integers(-50, ROWS + 50, 40).tolist(),
            "anything, many": rng.integers(-50, ROWS + 50, 400).tolist(), "sorted but for some": dented.tolist(), "falling": up[::-1].tolist()}


@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("pattern", list(patterns()))
def test_offsets_that_fall(torch, forced, pattern, kernel, gathered):  # noqa: F811
    offsets = np.array(patterns()[pattern], np.int64)
    E, N, K = len(offsets) - 1, 72, 640
    rng = np.random.default_rng(E)
    T = 45 if gathered else ROWS
    a, sa = R.random_operand(rng, T, K)
    b, sb = R.random_operand(rng, E * N, K, center=117)
    b, sb = b.reshape(E, N, -1), sb.reshape(E, N, -1)
    rows = rng.integers(0, T, ROWS).astype(np.int32)
    out, ok = guarded(torch, (ROWS, N), torch.float32)
    out.fill_(7.0)
    ta, tsa, tb, tsb, toff, trows = dev(torch, a, sa, b, sb, offsets.astype(np.int32), rows)
    forced(KERNELS[kernel])
    L.lpgemm_mxfp4_grouped(ta, tsa, tb, tsb, toff, rows=trows if gathered else None, out=out)
    assert ok()
    at = np.maximum.accumulate(offsets.clip(0, ROWS))
    x = R.values(a, sa)[rows if gathered else slice(None)]
    left = np.ones(ROWS, bool)
    for e in np.flatnonzero(at[1:] > at[:-1]):
        i, j = at[e], at[e + 1]
        held(out[i:j], x[i:j], R.values(b[e], sb[e]), "float32", f"group {e}")
        left[i:j] = False
    assert (out.cpu().numpy()[left] == 7.0).all()
