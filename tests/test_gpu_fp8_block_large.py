"""Block-scaled e4m3 operators at sizes whose offsets pass 32 bits, and on random
shapes (needs an MI355X)."""
import random

import numpy as np
import pytest

import fp8_block_reference as R
import precision_integer_gemm_amd as L
from test_gpu_fp8_block import codes_of, held, run_grouped, run_product, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def test_operand_past_32_bits(torch):  # noqa: F811
    """300000 rows of 8192 codes, 2.4 GB: the last rows as the first."""
    M, N, K = 300000, 40, 8192
    rng = np.random.default_rng(0)
    a, sa = R.random_operand(rng, 64, K)
    b, sb = R.random_operand(rng, N, K, 128)
    ta, tsa = (torch.from_numpy(v).cuda() for v in (a, sa))
    big = torch.zeros(M, K, dtype=torch.uint8, device="cuda")
    scales = torch.ones(M, K // 128, device="cuda")
    big[:64], big[-64:], scales[:64], scales[-64:] = ta, ta, tsa, tsa
    got = L.lpgemm_fp8_block(big, scales, torch.from_numpy(b).cuda(), torch.from_numpy(sb).cuda())
    held(got[:64], a, sa, b, sb, "bfloat16")
    assert torch.equal(got[:64], got[-64:]) and not got[64:-64].any()


def test_result_past_32_bits(torch):  # noqa: F811
    """70000 x 32768 results, 2.3e9 elements."""
    M, N, K = 70000, 32768, 128
    rng = np.random.default_rng(0)
    a, sa = R.random_operand(rng, M, K)
    b, sb = R.random_operand(rng, N, K, 128)
    got = L.lpgemm_fp8_block(*(torch.from_numpy(v).cuda() for v in (a, sa, b, sb)))
    for m, n in ((0, 0), (M - 50, N - 300), (65500, 100), (34000, 32000)):
        held(got[m:m + 50, n:n + 300], a[m:m + 50], sa[m:m + 50], b[n:n + 300], R.by_row(sb, N)[n:n + 300], "bfloat16", f"{m}, {n}")


def test_conversions_past_32_bits(torch):  # noqa: F811
    """300000 rows of 8192 values, 4.9 GB of bf16."""
    rows, K = 300000, 8192
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    part = torch.randn(200, K, device="cuda").bfloat16()
    x[:200], x[-200:] = part, part
    for block_rows in (1, 128):
        codes, scales = L.lpgemm_fp8_block_quantize(x, block_rows=block_rows)
        last = rows - 200
        first = -(-last // 128) * 128  # whole blocks of the last rows
        want_codes, want_scales = R.quantize(part[first - last:].float().cpu().numpy(), block_rows)
        np.testing.assert_array_equal(codes_of(codes[first:]), want_codes)
        np.testing.assert_array_equal(scales[first // block_rows:].cpu().numpy(), want_scales)
        back = L.lpgemm_fp8_block_dequantize(codes, scales, K)
        assert torch.equal(back[first:], L.lpgemm_fp8_block_dequantize(codes[first:].contiguous(), scales[first // block_rows:].contiguous(), K))
        assert not back[256:first - 128].any()


@pytest.mark.parametrize("seed", range(40))
def test_random_products(torch, seed):  # noqa: F811
    rng = random.Random(seed)
    M, N, K = (round(2 ** rng.uniform(0, t)) for t in (10, 11, 13))
    run_product(torch, M, N, K, rng.choice(("float32", "bfloat16", "float16")), rng.choice((1, 128)), seed)


@pytest.mark.parametrize("seed", range(30))
def test_random_groups(torch, seed):  # noqa: F811
    rng = random.Random(1000 + seed)
    E, N, K = (round(2 ** rng.uniform(0, t)) for t in (6, 10, 12))
    sizes = [round(2 ** rng.uniform(-1, rng.choice((3, 6, 9)))) for _ in range(E)]
    while sum(sizes) > 4000:
        sizes = [s // 2 for s in sizes]
    T = rng.randrange(1, 300)
    rows = np.random.default_rng(seed).integers(-1, T + 1, sum(sizes)) if rng.random() < 0.5 else None
    run_grouped(torch, np.random.default_rng(seed), sizes, N, K, rng.choice(("float32", "bfloat16")), rng.choice((1, 128)), T if rows is not None else None, rows)
