"""Conversions large enough for four items a thread and for passing by the
caches, every type, against calls of a few rows each (needs an MI355X)."""
import pytest

import precision_integer_gemm_amd as L
from test_gpu_mxfp4 import check_quantize, dtypes, guarded, torch  # noqa: F401

pytestmark = pytest.mark.gpu

# about 12, 60 and 110 million values: 2^20 items of eight and 192 MB lie between
SIZES = [(3001, 4099), (7001, 8500), (13001, 8448)]


@pytest.mark.parametrize("kind", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("rows,K", SIZES)
@pytest.mark.parametrize("gap", [0, 13])
def test_large(torch, kind, rows, K, gap):  # noqa: F811
    g = torch.Generator("cuda").manual_seed(rows + K)
    x = torch.empty(rows, K + gap, dtype=dtypes(torch)[kind], device="cuda").normal_(generator=g)[:, :K]
    U, step = -(-K // 128), 100
    codes, ok_c = guarded(torch, (rows, 64 * U), torch.uint8)
    scales, ok_s = guarded(torch, (rows, 4 * U), torch.uint8)
    y, ok_y = guarded(torch, (rows, K), dtypes(torch)[kind])
    L.lpgemm_mxfp4_quantize(x, codes=codes, scales=scales)
    L.lpgemm_mxfp4_dequantize(codes, scales, K, out=y)
    assert ok_c() and ok_s() and ok_y()
    for at in range(0, rows, step):
        i = slice(at, min(rows, at + step))
        c, s = L.lpgemm_mxfp4_quantize(x[i])
        assert torch.equal(codes[i], c) and torch.equal(scales[i], s), at
        assert torch.equal(y[i], L.lpgemm_mxfp4_dequantize(c, s, K, dtype=y.dtype)), at
    check_quantize(torch, x[rows - 60:])  # and one of those calls against the definition
