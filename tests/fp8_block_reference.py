"""e4m3 with a scale per block of 128 in numpy float64, written from its definition
and independent of the library: quantisation, values, products and the bounds
that the kernels are held to."""
import numpy as np

import fp8_bounds

BLOCK = 128
_c = np.arange(256)
_e, _m = (_c >> 3) & 15, _c & 7
VALUES = np.where(_e == 0, _m * 2.0 ** -9, (8 + _m) * np.exp2(_e - 10.0)) * np.where(_c & 128, -1, 1)
VALUES[[0x7F, 0xFF]] = np.nan


def units(K):
    return -(-K // BLOCK)


def encode(v):
    """Nearest code of float64 values up to 448, a tie going to the even code."""
    grid = VALUES[:127]
    a = np.abs(v)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    below, above = a - grid[hi - 1], grid[hi] - a
    code = np.where((below < above) | ((below == above) & (hi % 2 == 1)), hi - 1, hi)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def quantize(x, block_rows=1, power_of_two=False):
    """(codes uint8 [rows, 128 U], scales float32) of float32 rows, step by step in binary32."""
    rows, K = x.shape
    U, B = units(K), -(-rows // block_rows)
    p = np.zeros((B * block_rows, BLOCK * U), np.float32)
    p[:rows, :K] = x
    blocks = p.reshape(B, block_rows, U, BLOCK)
    with np.errstate(invalid="ignore"):
        a = np.abs(blocks).max((1, 3))
    fine = np.isfinite(a)
    low = np.maximum(np.where(fine, a, 1), np.float32(2.0 ** -100)).astype(np.float32)
    if power_of_two:
        e = np.frexp(low)[1] - 9.0
        e = np.where(low > 448 * np.exp2(e), e + 1, e)
        scale = np.exp2(e).astype(np.float32)
    else:
        scale = low / np.float32(448)
    inverse = np.float32(1) / scale
    y = np.where(fine[:, None, :, None], blocks, 0) * inverse[:, None, :, None]
    assert y.dtype == np.float32
    codes = encode(y.astype(np.float64)).reshape(B * block_rows, BLOCK * U)[:rows]
    codes = np.where(np.repeat(np.repeat(fine, block_rows, 0)[:rows], BLOCK, 1), codes, 0).astype(np.uint8)
    return codes, np.where(fine, scale, np.float32(np.nan)).astype(np.float32)


def by_row(scales, rows):
    """Scales of every row, given for each or for 128."""
    return scales if scales.shape[-2] == rows else np.repeat(scales, BLOCK, -2)[..., :rows, :]


def values(codes, scales):
    """float64 values, the padding included."""
    s = by_row(scales, codes.shape[-2]).astype(np.float64)
    return VALUES[codes] * np.repeat(s, BLOCK, -1)


def random_operand(rng, rows, K, block_rows=1, spread=4.0):
    """Random finite codes (half of them small) and scales of rows x K."""
    U = units(K)
    c = rng.integers(0, 256, (rows, BLOCK * U), dtype=np.uint8)
    c = np.where((c & 0x7F) == 0x7F, c & 0xF8, c)
    c = np.where(rng.random(c.shape) < 0.5, c & 0xBF, c).astype(np.uint8)
    c[:, K:] = 0
    s = np.exp2(rng.uniform(-8 - spread, -8 + spread, (-(-rows // block_rows), U))).astype(np.float32)
    return c, s


HALF_STEP = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
LEAST = {"float32": 2.0 ** -149, "bfloat16": 2.0 ** -133, "float16": 2.0 ** -24}


def product_bound(a, sa, b, sb, dtype):
    """(S, most |D - S|) of D = A B^T.  A block's sum from zero, one rounding of the
    scales' product, one fused step into the accumulator: U of these, and up to 8
    ranges of K added.  16-bit results: a group of 8 k is off by at most 7 2^(E - 13),
    a block by 16 group sums' roundings more; binary32 results: 128 additions of exact
    products.  Then one rounding to `dtype`."""
    va, vb = values(a, sa), values(b, sb)
    S, P = va @ vb.T, np.abs(va) @ np.abs(vb).T
    U = a.shape[1] // BLOCK
    if dtype == "float32":
        off = 1.01 * (U + 136) * 2.0 ** -24 * P
    else:
        off = 1.01 * (U + 24) * 2.0 ** -24 * P
        ra, rb = by_row(np.abs(sa).astype(np.float64), a.shape[0]), by_row(np.abs(sb).astype(np.float64), b.shape[0])
        for j in range(U):
            i = slice(BLOCK * j, BLOCK * (j + 1))
            off += fp8_bounds.group_exponent_bound(a[:, i], b[:, i], BLOCK) * ra[:, j:j + 1] * rb[:, j:j + 1].T
    return S, off + HALF_STEP[dtype] * (np.abs(S) + off) + LEAST[dtype]
