"""e4m3 operators with a scale per block of 128 against their definition in float64."""
import numpy as np
import pytest

import fp8_block_reference as R
import precision_integer_gemm_amd as L

pytestmark = pytest.mark.gpu
KINDS = ["float32", "bfloat16", "float16"]


@pytest.fixture(scope="module")
def torch():
    import torch
    return torch


def dtypes(torch):
    return {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


def dev(torch, *arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def guarded(torch, shape, dtype):
    """A tensor between two stretches of a pattern, and whether these are still whole."""
    n = int(np.prod(shape))
    buffer = torch.full((n + 512,), 3.0, dtype=dtype, device="cuda")
    return buffer[256:256 + n].view(shape), lambda: bool((buffer[:256] == 3).all()) and bool((buffer[256 + n:] == 3).all())


def codes_of(t):
    import torch
    return t.view(torch.uint8).cpu().numpy()


# ---- conversions -------------------------------------------------------------------
SIZES = [(1, 1), (1, 128), (3, 127), (2, 129), (127, 300), (128, 128), (129, 64), (5, 2897), (300, 40), (1, 8192), (1000, 640)]


def check_quantize(torch, x, block_rows, pow2):
    rows, K = x.shape
    shape = -(-rows // block_rows), R.units(K)
    codes, ok1 = guarded(torch, (rows, 128 * R.units(K)), torch.uint8)
    scales, ok2 = guarded(torch, shape, torch.float32)
    L.lpgemm_fp8_block_quantize(x, block_rows=block_rows, power_of_two=pow2, codes=codes, scales=scales)
    want, want_scales = R.quantize(x.float().cpu().numpy(), block_rows, pow2)
    assert ok1() and ok2()
    np.testing.assert_array_equal(scales.cpu().numpy(), want_scales)
    np.testing.assert_array_equal(codes.cpu().numpy(), want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("rows,K", SIZES)
def test_quantize(torch, kind, block_rows, pow2, rows, K):
    g = torch.Generator("cuda").manual_seed(rows * 31 + K)
    x = torch.randn(rows, K, device="cuda", generator=g) * torch.exp(2 * torch.randn(rows, 1, device="cuda", generator=g))
    check_quantize(torch, x.to(dtypes(torch)[kind]), block_rows, pow2)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_strided_rows(torch, kind, block_rows):
    x = torch.randn(300, 1000, device="cuda").to(dtypes(torch)[kind])
    for view in (x[:, 3:700], x[::3, 5:], x[7:8, 1:130], x[:, 999:]):
        check_quantize(torch, view, block_rows, False)


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
def test_quantize_every_exponent(torch, block_rows, pow2):
    """Blocks from the smallest subnormal to the largest finite value, zeros of both signs, the borders of 448."""
    rng = np.random.default_rng(0)
    e = np.arange(-149, 128)
    x = (rng.uniform(-1, 1, (e.size, 256)) * np.exp2(e.astype(np.float64))[:, None]).astype(np.float32)
    x[:, 0] = np.exp2(e)
    x[10] = 0
    x[11] = -0.0
    for i, v in enumerate((448, 464, 480, 1.75 * 2.0 ** 20, np.nextafter(np.float32(1.75), np.float32(2)))):
        x[20 + i, :128] = np.minimum(np.abs(x[20 + i, :128]), v)
        x[20 + i, 5] = v
    check_quantize(torch, torch.from_numpy(x).cuda(), block_rows, pow2)


@pytest.mark.parametrize("kind", ["bfloat16", "float16"])
def test_quantize_every_pattern(torch, kind):
    """All 65536 values of a 16-bit type; not finite ones take their block with them."""
    x = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(dtypes(torch)[kind])
    check_quantize(torch, x.view(-1, 256), 1, False)
    check_quantize(torch, x.view(256, -1).t().contiguous(), 1, True)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_not_finite(torch, block_rows):
    x = torch.randn(300, 400, device="cuda")
    x[3, 5], x[4, 140], x[200, 399], x[299, 0] = float("nan"), float("inf"), -float("inf"), float("nan")
    check_quantize(torch, x, block_rows, False)
    y = L.lpgemm_fp8_block_dequantize(*L.lpgemm_fp8_block_quantize(x, block_rows=block_rows), 400)
    want = torch.zeros(300, 400, dtype=torch.bool, device="cuda")
    for r, c in ((3, 0), (4, 128), (200, 384), (299, 0)):
        r0 = r // block_rows * block_rows
        want[r0:r0 + block_rows, c:c + 128] = True
    assert torch.equal(y.isnan(), want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,K", SIZES)
def test_dequantize(torch, kind, block_rows, rows, K):
    codes, scales = R.random_operand(np.random.default_rng(K), rows, K, block_rows)
    out, ok = guarded(torch, (rows, K), dtypes(torch)[kind])
    L.lpgemm_fp8_block_dequantize(*dev(torch, codes, scales), K, out=out)
    assert ok()
    v = R.VALUES[codes].astype(np.float32) * np.repeat(R.by_row(scales, rows), 128, 1)  # one rounding, then the type's
    want = torch.from_numpy(v[:, :K]).to(dtypes(torch)[kind])
    np.testing.assert_array_equal(out.cpu().float().numpy(), want.float().numpy())


def test_dequantize_every_code(torch):
    codes = np.arange(256, dtype=np.uint8).reshape(2, 128)
    got = L.lpgemm_fp8_block_dequantize(*dev(torch, codes, np.ones((2, 1), np.float32)), 128, dtype=torch.float32).cpu().numpy()
    np.testing.assert_array_equal(got, R.VALUES[codes].astype(np.float32))
    assert (np.signbit(got) == np.signbit(R.VALUES[codes]))[~np.isnan(got)].all()


def test_conversions_empty(torch):
    for shape in ((0, 100), (5, 0)):
        codes, scales = L.lpgemm_fp8_block_quantize(torch.zeros(shape, device="cuda"))
        assert codes.shape == (shape[0], 128 * R.units(shape[1])) and scales.shape == (shape[0], R.units(shape[1]))
        assert L.lpgemm_fp8_block_dequantize(codes, scales, shape[1]).shape == shape


# ---- the product -----------------------------------------------------------------------
def held(got, a, sa, b, sb, kind, what=""):
    S, bound = R.product_bound(a, sa, b, sb, kind)
    off = np.abs(got.double().cpu().numpy() - S)
    assert np.isfinite(off).all(), what
    worst = (off / np.maximum(bound, 1e-300)).max(initial=0)
    assert worst <= 1, f"{what}: {worst} of the bound"


def run_product(torch, M, N, K, kind, block_rows, seed=0):
    rng = np.random.default_rng(M * 7 + N * 3 + K + seed)
    a, sa = R.random_operand(rng, M, K)
    b, sb = R.random_operand(rng, N, K, block_rows)
    out, ok = guarded(torch, (M, N), dtypes(torch)[kind])
    L.lpgemm_fp8_block(*dev(torch, a, sa, b, sb), out=out)
    assert ok()
    held(out, a, sa, b, sb, kind)


PRODUCTS = [(1, 1, 1), (1, 1024, 4096), (2, 33, 31), (5, 64, 128), (16, 1000, 2897), (17, 257, 640), (31, 128, 8192), (33, 4, 4100),
            (64, 512, 1024), (65, 77, 129), (100, 700, 257), (128, 128, 384), (129, 1001, 512), (200, 3, 3000), (255, 300, 1200),
            (256, 256, 256), (333, 1001, 2897), (513, 770, 900), (16, 333, 16384), (48, 40, 20000), (7, 50, 9000), (700, 1304, 128)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(torch, kind, block_rows, M, N, K):
    run_product(torch, M, N, K, kind, block_rows)


KERNELS = {"64": L.KERNEL_TILED_64, "128": L.KERNEL_TILED_128, "256": L.KERNEL_TILED_256, "skinny": L.KERNEL_SKINNY}


@pytest.fixture(params=list(KERNELS))
def forced(request):
    L.lpgemm_set_kernel_override(KERNELS[request.param])
    yield request.param
    L.lpgemm_set_kernel_override(L.KERNEL_AUTO)


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("M,N,K", [(1, 5, 1), (40, 70, 300), (130, 260, 640), (300, 513, 2200), (257, 140, 9000), (65, 1, 16500)])
def test_every_kernel(torch, forced, kind, block_rows, M, N, K):
    run_product(torch, M, N, K, kind, block_rows, seed=5)


@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
def test_every_unit_counts(torch, forced, kind):
    """Every block of every row has its own scales and its own value of k, K long and ragged."""
    M, N, K = 70, 150, 1300
    U = R.units(K)
    rng = np.random.default_rng(1)
    a, b = np.zeros((M, 128 * U), np.uint8), np.zeros((N, 128 * U), np.uint8)
    for i in range(M):
        j = i % U
        a[i, min(128 * j + (37 * i) % 128, K - 1)] = 0x38 + i % 8
    b[:, :K] = rng.integers(0x30, 0x48, (N, K))
    sa, sb = np.exp2(rng.integers(-3, 4, (M, U))).astype(np.float32), np.exp2(rng.integers(-3, 4, (N, U))).astype(np.float32)
    got = L.lpgemm_fp8_block(*dev(torch, a, sa, b, sb), dtype=dtypes(torch)[kind]).cpu()
    want = torch.from_numpy(R.values(a, sa) @ R.values(b, sb).T).to(dtypes(torch)[kind])  # one product each: exact
    assert torch.equal(got, want)


@pytest.mark.parametrize("M,N,K", [(1, 64, 512), (16, 100, 300), (40, 300, 4096), (300, 300, 640)])
def test_product_nan_scales_and_codes(torch, M, N, K):
    rng = np.random.default_rng(M)
    a, sa = R.random_operand(rng, M, K)
    b, sb = R.random_operand(rng, N, K)
    sa[M // 2, 1] = np.nan
    sb[N // 3, 2] = np.nan
    b[N // 2, 7] = 0x7F
    got = L.lpgemm_fp8_block(*dev(torch, a, sa, b, sb)).float().cpu().numpy()
    want = np.zeros((M, N), bool)
    want[M // 2], want[:, N // 3], want[:, N // 2] = True, True, True
    np.testing.assert_array_equal(np.isnan(got), want)


@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_product_scales_far_apart(torch, M):
    """Blocks from 2^-60 to 2^60 against the other side's opposite."""
    rng = np.random.default_rng(M)
    a, sa = R.random_operand(rng, M, 1024)
    b, sb = R.random_operand(rng, 100, 1024)
    e = rng.integers(-60, 61, sa.shape[1])
    sa, sb = (sa * np.exp2(e)).astype(np.float32), (sb * np.exp2(-e)).astype(np.float32)
    for kind in KINDS:
        held(L.lpgemm_fp8_block(*dev(torch, a, sa, b, sb), dtype=dtypes(torch)[kind]), a, sa, b, sb, kind)


@pytest.mark.parametrize("M", [1, 3, 16, 17, 40, 130, 300])
def test_product_same_bits_again(torch, M):
    rng = np.random.default_rng(M)
    a, sa = R.random_operand(rng, M, 8192)
    b, sb = R.random_operand(rng, 512, 8192, 128)
    t = dev(torch, a, sa, b, sb)
    first = L.lpgemm_fp8_block(*t, dtype=torch.bfloat16)
    for _ in range(3):
        assert torch.equal(L.lpgemm_fp8_block(*t, dtype=torch.bfloat16), first)


def test_product_empty(torch):
    c = lambda *s: torch.zeros(s, dtype=torch.float8_e4m3fn, device="cuda")  # noqa: E731
    f = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    assert L.lpgemm_fp8_block(c(0, 128), f(0, 1), c(5, 128), f(5, 1)).shape == (0, 5)
    assert L.lpgemm_fp8_block(c(5, 128), f(5, 1), c(0, 128), f(0, 1)).shape == (5, 0)
    out = torch.full((5, 6), 3.0, device="cuda")
    L.lpgemm_fp8_block(c(5, 0), f(5, 0), c(6, 0), f(6, 0), out=out)
    assert not out.any()


# ---- grouped -----------------------------------------------------------------------------
def run_grouped(torch, rng, sizes, N, K, kind, block_rows=128, T=None, rows=None):
    E, R_ = len(sizes), int(np.sum(sizes)) if rows is None else len(rows)
    T = R_ if T is None else T
    a, sa = R.random_operand(rng, T, K)
    made = [R.random_operand(rng, N, K, block_rows) for _ in range(E)]
    b, sb = np.stack([m[0] for m in made]), np.stack([m[1] for m in made])
    offsets = np.concatenate(([0], np.cumsum(sizes))).astype(np.int32)
    out, ok = guarded(torch, (R_, N), dtypes(torch)[kind])
    out.fill_(7.0)
    ta, tsa, tb, tsb, toff = dev(torch, a, sa, b, sb, offsets)
    trows = None if rows is None else dev(torch, np.asarray(rows, np.int32))[0]
    L.lpgemm_fp8_block_grouped(ta, tsa, tb, tsb, toff, rows=trows, out=out)
    assert ok()
    at = np.arange(R_) if rows is None else np.asarray(rows, np.int64)
    there = ((at >= 0) & (at < T))[:, None]
    at = at.clip(0, max(T - 1, 0))
    x = np.where(there, a[at], 0) if T else np.zeros((R_, a.shape[1]), np.uint8)
    sx = np.where(there, sa[at], 0) if T else np.zeros((R_, sa.shape[1]), np.float32)
    for e in range(E):
        i, j = offsets[e], offsets[e + 1]
        if j > i:
            held(out[i:j], x[i:j], sx[i:j], b[e], sb[e], kind, f"group {e}")
    assert (out[int(offsets[-1]):] == 7).all()
    return out


SPLITS = {"one": [40], "even": [16] * 5, "single rows": [1] * 33, "empty ones": [0, 5, 0, 0, 33, 1, 0], "all empty": [0, 0, 0],
          "skewed": [300, 1, 0, 7, 64, 2], "tile edges": [31, 32, 33, 127, 128, 129, 255, 256, 257], "many": [3, 0, 1, 9] * 32,
          "one large": [0, 0, 700, 0]}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("split", list(SPLITS))
@pytest.mark.parametrize("N,K,block_rows", [(96, 512, 1), (301, 1897, 128), (8, 40, 128)])
def test_grouped(torch, kind, split, N, K, block_rows):
    run_grouped(torch, np.random.default_rng(N), SPLITS[split], N, K, kind, block_rows)


@pytest.mark.parametrize("split", ["single rows", "empty ones", "skewed", "tile edges", "many"])
@pytest.mark.parametrize("kind", ["float32", "bfloat16"])
def test_grouped_gathered_rows(torch, split, kind):
    """Rows taken through an index, some of them many times, some outside A (zeros)."""
    rng = np.random.default_rng(8)
    n = int(np.sum(SPLITS[split]))
    rows = rng.integers(0, 50, n)
    rows[::7] = -1
    rows[3::11] = 50
    rows[5::13] = 2 ** 31 - 1
    rows[6::17] = -2 ** 31
    out = run_grouped(torch, rng, SPLITS[split], 200, 700, kind, T=50, rows=rows)
    assert not out[::7].any()


@pytest.mark.parametrize("sizes", [[33, 0, 97], [5, 2, 0, 1]])
def test_grouped_every_kernel(torch, forced, sizes):
    rows = np.random.default_rng(3).integers(0, 20, int(np.sum(sizes)))
    run_grouped(torch, np.random.default_rng(4), sizes, 150, 1700, "bfloat16", T=20, rows=rows)
    run_grouped(torch, np.random.default_rng(5), sizes, 270, 600, "float32", 1)


def test_grouped_no_rows_of_a(torch):
    assert not run_grouped(torch, np.random.default_rng(0), [3, 2], 64, 256, "float32", T=0, rows=[0, 1, -1, 5, 0]).any()


def test_grouped_rows_in_no_group_stay(torch):
    rng = np.random.default_rng(4)
    a, sa = R.random_operand(rng, 60, 256)
    made = [R.random_operand(rng, 40, 256, 128) for _ in range(3)]
    b, sb = np.stack([m[0] for m in made]), np.stack([m[1] for m in made])
    t = dev(torch, a, sa, b, sb)
    for offsets, groups in (([5, 20, 20, 50], [(5, 20), None, (20, 50)]), ([-7, 10, 30, 99], [(0, 10), (10, 30), (30, 60)]),
                            ([0, 40, 20, 20], [(0, 40), None, None]), ([70, 80, 90, 100], [None] * 3),
                            ([-2 ** 31, 2 ** 31 - 1, 0, 0], [(0, 60), None, None])):
        out, ok = guarded(torch, (60, 40), torch.float32)
        out.fill_(7.0)
        L.lpgemm_fp8_block_grouped(*t, dev(torch, np.array(offsets, np.int32))[0], out=out)
        assert ok()
        left = np.ones(60, bool)
        for e, g in enumerate(groups):
            if g:
                held(out[g[0]:g[1]], a[g[0]:g[1]], sa[g[0]:g[1]], b[e], sb[e], "float32")
                left[g[0]:g[1]] = False
        assert (out.cpu().numpy()[left] == 7.0).all()


# ---- a linear layer's three products -------------------------------------------------------
def test_linear_layer_gradients(torch):
    """y = x w^T, its input's gradient from the transposed codes and scales, its weight's from both sides quantised
    along the tokens: each within its operands' bound, so the transposed weight is the same weight."""
    T, N, K = 200, 384, 512
    g = torch.Generator("cuda").manual_seed(0)
    x, dy = torch.randn(T, K, device="cuda", generator=g), torch.randn(T, N, device="cuda", generator=g)
    w = torch.randn(N, K, device="cuda", generator=g) / K ** 0.5
    q = L.lpgemm_fp8_block_quantize
    wc, ws = q(w, block_rows=128)
    pairs = {"y": (*q(x), wc, ws), "dx": (*q(dy), wc.t().contiguous(), ws.t().contiguous()), "dw": (*q(dy.t().contiguous()), *q(x.t().contiguous()))}
    exact = {"y": x.double() @ w.double().t(), "dx": dy.double() @ w.double(), "dw": dy.double().t() @ x.double()}
    for name, p in pairs.items():
        got = L.lpgemm_fp8_block(*p, dtype=torch.float32)
        held(got, codes_of(p[0]), p[1].cpu().numpy(), codes_of(p[2]), p[3].cpu().numpy(), "float32", name)
        # each operand is off by at most 2^-4 of a value: independent errors, so far less of the whole
        assert float((got - exact[name]).norm() / exact[name].norm()) < 2.0 ** -4, name


# ---- streams and graphs ----------------------------------------------------------------------
def chain(torch, x, w, sw, offsets, rows):
    codes, scales = L.lpgemm_fp8_block_quantize(x)
    y = L.lpgemm_fp8_block_grouped(codes, scales, w, sw, offsets, rows=rows, dtype=torch.bfloat16)
    z = L.lpgemm_fp8_block(codes, scales, w[0], sw[0], dtype=torch.float32)
    return y, z, L.lpgemm_fp8_block_dequantize(codes, scales, x.shape[1])


@pytest.fixture(params=[(24, 1024), (300, 640), (2, 8192)])
def chained(torch, request):
    T, K = request.param
    rng = np.random.default_rng(T)
    made = [R.random_operand(rng, 96, K, 128) for _ in range(4)]
    w, sw = dev(torch, np.stack([m[0] for m in made]), np.stack([m[1] for m in made]))
    offsets, rows = dev(torch, np.array([0, T // 2, T // 2, T, 2 * T], np.int32), rng.integers(0, T, 2 * T).astype(np.int32))
    return torch.randn(T, K, device="cuda"), w, sw, offsets, rows


def test_another_stream(torch, chained):
    want = chain(torch, *chained)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = chain(torch, *chained)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x, w, sw, offsets, rows = chained
    codes, scales = L.lpgemm_fp8_block_quantize(x, stream=s)
    y = L.lpgemm_fp8_block_grouped(codes, scales, w, sw, offsets, rows=rows, stream=s)
    s.synchronize()
    assert torch.equal(y, want[0])


def test_graph_replays(torch, chained):
    x, *rest = chained
    static = x.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        chain(torch, static, *rest)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(torch, static, *rest)
    for seed in range(4):
        new = torch.randn(x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
        static.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        want = chain(torch, new, *rest)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), seed
