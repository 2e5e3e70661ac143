"""The microscaled 4-bit format in numpy float64, written from its definition
and independent of the library: quantisation, values, products and the bounds
that the kernels are held to."""
import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
UNIT = 128


def units(K):
    return -(-K // UNIT)


def quantize(x):
    """(codes uint8 [rows, 64 U], scales uint8 [rows, 4 U]) of float64 rows."""
    rows, K = x.shape
    U = units(K)
    codes = np.zeros((rows, UNIT * U), np.uint8)
    scales = np.full((rows, 4 * U), 127, np.uint8)
    for j in range(-(-K // 32)):
        b = x[:, 32 * j:32 * j + 32]
        fine = np.isfinite(b).all(1)
        a = np.where(fine, np.abs(np.where(np.isfinite(b), b, 0)).max(1), 0)
        e = np.where(a > 0, np.frexp(a)[1] - 3, -127).clip(-127, None)
        v = np.ldexp(np.where(fine[:, None], b, 0), -e[:, None])
        # nearest grid value: the distance decides, a tie goes to the even code
        d = np.abs(np.minimum(np.abs(v), 6)[:, :, None] - GRID)
        best = d.min(2, keepdims=True)
        tied = d == best
        first = tied.argmax(2)
        last = 7 - tied[:, :, ::-1].argmax(2)
        code = np.where(first % 2 == 0, first, last)
        codes[:, 32 * j:32 * j + b.shape[1]] = np.where(fine[:, None], code + 8 * np.signbit(b), 0)
        scales[:, j] = np.where(fine, e + 127, 255)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales


def values(codes, scales):
    """float64 values, the padding included; a scale of 255 gives NaN."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = np.where(c & 8, -1.0, 1.0) * GRID[c & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return v * np.repeat(s, 32, -1)


def random_operand(rng, rows, K, spread=6, center=121):
    """Random codes and scales of rows x K, the padding as the format wants it."""
    U = units(K)
    c = rng.integers(0, 16, (rows, UNIT * U), dtype=np.uint8)
    c[:, K:] = 0
    s = rng.integers(center - spread, center + spread + 1, (rows, 4 * U), dtype=np.uint8)
    s[:, -(-K // 32):] = 127
    return c[:, 0::2] | (c[:, 1::2] << 4), s


# half a step of each result type, relative to the value, and its least step
HALF_STEP = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
LEAST = {"float32": 2.0 ** -149, "bfloat16": 2.0 ** -133, "float16": 2.0 ** -24}


def product_bound(va, vb, dtype):
    """(S, most |D - S|) for operands' values: binary32 sums of exact groups of
    8 products, at most K / 8 + 16 additions, each off by at most 2^-24 of a
    partial sum that is below P = sum |a b|; then one rounding to `dtype`."""
    S = va @ vb.T
    P = np.abs(va) @ np.abs(vb).T
    off = 1.01 * (va.shape[1] / 8 + 16) * 2.0 ** -24 * P
    return S, off + HALF_STEP[dtype] * (np.abs(S) + off) + LEAST[dtype]
