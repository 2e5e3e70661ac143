"""Conversions of more rows than one launch holds (needs an MI355X): 2^32
threads are 2^30 rows of one unit."""
import pytest

import precision_integer_gemm_amd as L
from test_gpu_mxfp4 import torch  # noqa: F401

pytestmark = pytest.mark.gpu


def test_more_rows_than_a_launch_holds(torch):  # noqa: F811
    rows, border = (1 << 30) + 100, (1 << 30) - 64
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of device memory")
    x = torch.empty(rows, 2, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(0))[:, :1]
    codes = torch.full((rows, 64), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, 4), 0xA5, dtype=torch.uint8, device="cuda")
    L.lpgemm_mxfp4_quantize(x, codes=codes, scales=scales)
    y = torch.full((rows, 1), 9.0, dtype=torch.bfloat16, device="cuda")
    L.lpgemm_mxfp4_dequantize(codes, scales, 1, out=y)
    for at in (0, 1 << 20, (1 << 29) - 50, border - 100, border - 1, border, rows - 100):
        i = slice(at, min(rows, at + 100))
        c, s = L.lpgemm_mxfp4_quantize(x[i])
        assert torch.equal(codes[i], c) and torch.equal(scales[i], s), at
        assert torch.equal(y[i], L.lpgemm_mxfp4_dequantize(c, s, 1)), at
    # alone in its block a value lies in [4, 8) scales and becomes 4 or 6: off by less than a quarter of itself
    for at in range(0, rows, 1 << 27):
        i = slice(at, min(rows, at + (1 << 27)))
        assert bool(((y[i] - x[i]).abs() <= x[i].abs() / 4).all()), at
    del x, y, codes, scales
    torch.cuda.empty_cache()
