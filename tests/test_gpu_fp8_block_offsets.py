"""Offsets of the grouped block-scaled product that fall somewhere (needs an
MI355X): an offset below one before it counts as that one, so every row has one
group at most, whatever the offsets hold."""
import numpy as np
import pytest

import fp8_block_reference as R
import precision_integer_gemm_amd as L
from test_gpu_fp8_block import dev, dtypes, guarded, held, torch  # noqa: F401
from test_gpu_mxfp4_offsets import KERNELS, ROWS, patterns  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture
def force():
    yield L.lpgemm_set_kernel_override
    L.lpgemm_set_kernel_override(L.KERNEL_AUTO)


@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("pattern", list(patterns()))
def test_offsets_that_fall(torch, force, pattern, kernel, gathered):  # noqa: F811
    offsets = np.array(patterns()[pattern], np.int64)
    E, N, K = len(offsets) - 1, 72, 640
    rng = np.random.default_rng(E)
    T = 45 if gathered else ROWS
    a, sa = R.random_operand(rng, T, K)
    b, _ = R.random_operand(rng, E * N, K)
    b, sb = b.reshape(E, N, -1), np.exp2(rng.uniform(-12, -4, (E, 1, K // 128))).astype(np.float32)
    rows = rng.integers(0, T, ROWS).astype(np.int32)
    out, ok = guarded(torch, (ROWS, N), torch.bfloat16)
    out.fill_(7.0)
    ta, tsa, tb, tsb, toff, trows = dev(torch, a, sa, b, sb, offsets.astype(np.int32), rows)
    force(KERNELS[kernel])
    L.lpgemm_fp8_block_grouped(ta, tsa, tb, tsb, toff, rows=trows if gathered else None, out=out)
    assert ok()
    at = np.maximum.accumulate(offsets.clip(0, ROWS))
    x, sx = (a[rows], sa[rows]) if gathered else (a, sa)
    left = np.ones(ROWS, bool)
    for e in np.flatnonzero(at[1:] > at[:-1]):
        i, j = at[e], at[e + 1]
        held(out[i:j], x[i:j], sx[i:j], b[e], sb[e], "bfloat16", f"group {e}")
        left[i:j] = False
    assert (out.float().cpu().numpy()[left] == 7.0).all()
