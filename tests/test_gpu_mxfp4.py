"""The microscaled 4-bit operators on the GPU against their definition in
float64 (needs an MI355X).

Quantisation and dequantisation are held to equality.  A product is held to
the bound of binary32 sums of exact groups of eight products (mxfp4_reference.
product_bound): the kernels may add in any order, so every kernel and split
has the same bound.  Results sit between guard bands.
"""
import numpy as np
import pytest

import mxfp4_reference as R
import precision_integer_gemm_amd as L

pytestmark = pytest.mark.gpu

GUARD = 512


@pytest.fixture(scope="module")
def torch():
    import torch as t
    if not t.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()
    return t


def dtypes(torch):
    return {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}


def guarded(torch, shape, dtype):
    """A dense tensor of `shape` inside a buffer of sentinels, and a check that they are still there."""
    n = int(np.prod(shape))
    buf = torch.empty(n + 2 * GUARD, dtype=dtype, device="cuda")
    bits = buf.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[buf.element_size()])
    bits.fill_(0x5A)

    def untouched():
        return bool((bits[:GUARD] == 0x5A).all()) and bool((bits[GUARD + n:] == 0x5A).all())
    return buf[GUARD:GUARD + n].view(shape), untouched


def dev(torch, *arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def check_quantize(torch, x):
    """x: a tensor on the device (possibly strided)."""
    rows, K = x.shape
    U = R.units(K)
    codes, ok_c = guarded(torch, (rows, 64 * U), torch.uint8)
    scales, ok_s = guarded(torch, (rows, 4 * U), torch.uint8)
    L.lpgemm_mxfp4_quantize(x, codes=codes, scales=scales)
    want_c, want_s = R.quantize(x.double().cpu().numpy())
    got_s, got_c = scales.cpu().numpy(), codes.cpu().numpy()
    assert ok_c() and ok_s()
    np.testing.assert_array_equal(got_s, want_s)
    np.testing.assert_array_equal(got_c, want_c)


# ---- quantisation ------------------------------------------------------------
@pytest.mark.parametrize("kind", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 8192), (3, 31), (2, 32), (5, 33), (7, 127), (4, 128), (3, 129), (70, 1000),
                                    (33, 4101), (2, 16384), (300, 40)])
def test_quantize(torch, kind, rows, K):
    g = torch.Generator("cuda").manual_seed(rows * 100003 + K)
    x = torch.randn(rows, K, device="cuda", generator=g) * torch.exp(2 * torch.randn(rows, 1, device="cuda", generator=g))
    x[torch.rand(rows, K, device="cuda", generator=g) < 0.1] = 0
    check_quantize(torch, x.to(dtypes(torch)[kind]))


@pytest.mark.parametrize("kind", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("start,K,stride", [(0, 2897, 2913), (1, 128, 131), (3, 500, 512), (8, 256, 264), (5, 77, 1000)])
def test_quantize_strided_rows(torch, kind, start, K, stride):
    x = torch.randn(37, stride + 8, device="cuda", generator=torch.Generator("cuda").manual_seed(K)).to(dtypes(torch)[kind])
    base = x.view(-1)[start:start + 36 * stride + K]
    check_quantize(torch, base.as_strided((37, K), (stride, 1), base.storage_offset()))


@pytest.mark.parametrize("partner", [None, -3, 0, 1, 2, 3, 4, 30])
def test_quantize_every_bfloat16(torch, partner):
    """Every bf16 value, alone in its block or beside one of 2^partner times its binade: all scales, all ties."""
    bits = np.arange(65536, dtype=np.uint32)
    v = (bits << 16).view(np.float32)
    x = np.zeros((65536, 32), np.float32)
    x[:, 17] = v
    if partner is not None:
        with np.errstate(over="ignore", invalid="ignore"):
            x[:, 4] = np.where(np.isfinite(v), np.ldexp(np.float32(1.5), np.clip(np.frexp(np.abs(v))[1] - 1 + partner, -133, 126)), 0)
    x = x.reshape(-1, 4096)
    check_quantize(torch, torch.from_numpy(x).cuda().to(torch.bfloat16))


def test_quantize_every_float16(torch):
    bits = np.arange(65536, dtype=np.uint16)
    x = np.zeros((65536, 32), np.float16)
    x[:, 9] = bits.view(np.float16)
    x[:, 30] = np.roll(bits, 1).view(np.float16)
    check_quantize(torch, torch.from_numpy(x.reshape(-1, 2048)).cuda())


def test_quantize_every_bfloat16_among_others(torch):
    """Every pair of neighbouring bf16 patterns packed as they come: blocks of one binade."""
    x = np.arange(65536, dtype=np.uint32) << 16
    check_quantize(torch, torch.from_numpy(x.view(np.float32).reshape(16, 4096)).cuda().to(torch.bfloat16))


@pytest.mark.parametrize("kind", ["float32", "bfloat16", "float16"])
def test_quantize_ties_in_every_place(torch, kind):
    """Each border of the grid and its neighbours, both signs, in every place of a block, at several scales."""
    step = {"float32": 2.0 ** -23, "bfloat16": 2.0 ** -7, "float16": 2.0 ** -10}[kind]
    borders = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0])
    rows = []
    for power in (-9, 0, 5):
        for at in range(32):
            for f in (1 - step, 1.0, 1 + step):
                x = np.zeros((18, 32))
                x[:, at] = np.concatenate((borders, -borders)) * f
                x[:, (at + 7) % 32] = 4.0
                rows.append(np.ldexp(x, power))
    x = np.concatenate(rows).reshape(-1, 64)
    check_quantize(torch, torch.from_numpy(x).cuda().to(dtypes(torch)[kind]))


def test_quantize_extremes_float32(torch):
    rng = np.random.default_rng(3)
    x = np.ldexp(rng.uniform(-2, 2, (64, 256)), rng.integers(-151, 128, (64, 8)).repeat(32, 1))
    x = np.where(np.abs(x) > 3.4e38, 3.4e38, x).astype(np.float32)
    x[3, 5], x[4, 40], x[5, 255], x[6, 100] = np.nan, np.inf, -np.inf, -0.0
    x[7] = 0
    x[8] = -0.0
    check_quantize(torch, torch.from_numpy(x).cuda())


def test_quantize_empty(torch):
    for shape in ((0, 100), (5, 0)):
        codes, scales = L.lpgemm_mxfp4_quantize(torch.zeros(shape, device="cuda"))
        assert codes.shape == (shape[0], 64 * R.units(shape[1])) and scales.shape == (shape[0], 4 * R.units(shape[1]))


# ---- dequantisation ----------------------------------------------------------
@pytest.mark.parametrize("kind", ["float32", "bfloat16", "float16"])
def test_dequantize_every_code_and_scale(torch, kind):
    codes = np.tile(np.arange(256, dtype=np.uint8).reshape(16, 16), (256, 1)).reshape(-1, 64)  # 256 blocks of 16 rows
    scales = np.arange(256, dtype=np.uint8).repeat(16).reshape(-1, 4)
    c, s = dev(torch, codes, scales)
    got = L.lpgemm_mxfp4_dequantize(c, s, 128, dtype=dtypes(torch)[kind])
    v = R.values(codes, scales)
    want = torch.from_numpy(v).to(torch.float32 if kind != "float16" else torch.float16)  # one rounding at most
    if kind == "bfloat16":
        want = want.to(torch.bfloat16)
    np.testing.assert_array_equal(got.cpu().float().numpy(), want.float().numpy())
    assert (np.signbit(got.cpu().float().numpy()) == np.signbit(v))[~np.isnan(v)].all()


@pytest.mark.parametrize("kind", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 31), (2, 129), (5, 2897), (1, 8192), (300, 40)])
def test_dequantize_sizes(torch, kind, rows, K):
    codes, scales = R.random_operand(np.random.default_rng(K), rows, K)
    out, ok = guarded(torch, (rows, K), dtypes(torch)[kind])
    L.lpgemm_mxfp4_dequantize(*dev(torch, codes, scales), K, out=out)
    assert ok()
    want = torch.from_numpy(R.values(codes, scales)[:, :K]).to(dtypes(torch)[kind])
    np.testing.assert_array_equal(out.cpu().float().numpy(), want.float().numpy())


# ---- the product ---------------------------------------------------------------
def held(got, va, vb, kind, what=""):
    S, bound = R.product_bound(va, vb, kind)
    off = np.abs(got.double().cpu().numpy() - S)
    assert np.isfinite(off).all(), what
    worst = (off / np.maximum(bound, 1e-300)).max(initial=0)
    assert worst <= 1, f"{what}: {worst} of the bound"


SIZES = [(1, 1, 1), (1, 4096, 4096), (2, 33, 31), (5, 64, 128), (16, 1000, 2897), (17, 257, 640), (31, 128, 8192), (33, 4, 4100),
         (64, 512, 1024), (65, 77, 129), (100, 2048, 257), (128, 128, 384), (129, 1001, 512), (200, 3, 3000), (255, 300, 1200),
         (256, 256, 256), (333, 1001, 2897), (513, 770, 900), (1000, 1100, 640), (1, 28672, 512), (16, 3333, 16384), (48, 40, 40000),
         (700, 2304, 128)]


@pytest.mark.parametrize("kind", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(torch, kind, M, N, K):
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    a, sa = R.random_operand(rng, M, K)
    b, sb = R.random_operand(rng, N, K, center=117)
    out, ok = guarded(torch, (M, N), dtypes(torch)[kind])
    L.lpgemm_mxfp4(*dev(torch, a, sa, b, sb), out=out)
    assert ok()
    held(out, R.values(a, sa), R.values(b, sb), kind)


@pytest.mark.parametrize("M", [1, 3, 16, 17, 40, 70, 130, 300])
def test_product_same_bits_again(torch, M):
    """No order of additions that changes from call to call; the workspace's old contents do not matter."""
    rng = np.random.default_rng(M)
    a, sa = R.random_operand(rng, M, 8192)
    b, sb = R.random_operand(rng, 512, 8192)
    t = dev(torch, a, sa, b, sb)
    first = L.lpgemm_mxfp4(*t, dtype=torch.float32)
    for fill in (0xFF, 0x00, 0x7B):
        ws = torch.full((max(1, L.lpgemm_mxfp4_workspace_size(M, 512, 8192)) + 256,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(L.lpgemm_mxfp4(*t, dtype=torch.float32, workspace=ws), first)
    held(L.lpgemm_mxfp4(*t, dtype=torch.float32, workspace=None), R.values(a, sa), R.values(b, sb), "float32", "no workspace")
    small = torch.empty(512, dtype=torch.uint8, device="cuda")
    held(L.lpgemm_mxfp4(*t, dtype=torch.float32, workspace=small), R.values(a, sa), R.values(b, sb), "float32", "a small workspace")


@pytest.mark.parametrize("M,N", [(3, 40), (40, 70), (300, 300)])
def test_product_every_k_counts(torch, M, N):
    """One k at a time: D is that k's column of A times B's, whatever kernel and place."""
    K = 700
    rng = np.random.default_rng(1)
    b, sb = R.random_operand(rng, N, K)
    vb = R.values(b, sb)
    x = np.zeros((M, K), np.float32)
    for i in range(M):
        x[i, (i * 37 + 5) % K] = 1.5
    a, sa = R.quantize(x.astype(np.float64))
    got = L.lpgemm_mxfp4(*dev(torch, a, sa, b, sb), dtype=torch.float32).cpu().numpy()
    np.testing.assert_array_equal(got, (R.values(a, sa) @ vb.T).astype(np.float32))


@pytest.mark.parametrize("M,N", [(1, 64), (16, 100), (40, 70), (300, 300)])
def test_product_scales_at_their_ends(torch, M, N):
    """Scales from 2^-60 to 2^60 against each other, rows and blocks far apart."""
    K = 1024
    rng = np.random.default_rng(M)
    a, sa = R.random_operand(rng, M, K)
    b, sb = R.random_operand(rng, N, K)
    sa = rng.integers(127 - 55, 127 + 55, (M, 1), dtype=np.uint8) + rng.integers(0, 5, sa.shape, dtype=np.uint8)
    sb = rng.integers(127 - 5, 127 + 5, (N, 1), dtype=np.uint8) + rng.integers(0, 5, sb.shape, dtype=np.uint8)
    got = L.lpgemm_mxfp4(*dev(torch, a, sa, b, sb), dtype=torch.float32)
    held(got, R.values(a, sa), R.values(b, sb), "float32")


@pytest.mark.parametrize("M,N,K", [(1, 64, 512), (16, 100, 300), (40, 70, 4096), (300, 300, 640)])
def test_product_nan_scale(torch, M, N, K):
    rng = np.random.default_rng(M)
    a, sa = R.random_operand(rng, M, K)
    b, sb = R.random_operand(rng, N, K)
    sa[M // 2, 1] = 255
    sb[N // 3, 3] = 255
    got = L.lpgemm_mxfp4(*dev(torch, a, sa, b, sb), dtype=torch.bfloat16).float().cpu().numpy()
    want = np.zeros((M, N), bool)
    want[M // 2], want[:, N // 3] = True, True
    np.testing.assert_array_equal(np.isnan(got), want)


def test_product_empty(torch):
    z = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    assert L.lpgemm_mxfp4(z(0, 64), z(0, 4), z(5, 64), z(5, 4)).shape == (0, 5)
    assert L.lpgemm_mxfp4(z(5, 64), z(5, 4), z(0, 64), z(0, 4)).shape == (5, 0)
    out = torch.full((5, 6), 3.0, device="cuda")
    L.lpgemm_mxfp4(z(5, 0), z(5, 0), z(6, 0), z(6, 0), out=out)
    assert not out.any()


# ---- grouped ---------------------------------------------------------------------
def run_grouped(torch, rng, sizes, N, K, kind, T=None, rows=None, cover=None):
    """Result (a numpy array), its groups' slices and the operands' values."""
    E, R_ = len(sizes), int(np.sum(sizes)) if rows is None else len(rows)
    T = R_ if T is None else T
    a, sa = R.random_operand(rng, T, K)
    b, sb = R.random_operand(rng, max(1, E * N), K, center=117)
    b, sb = b[:E * N].reshape(E, N, -1), sb[:E * N].reshape(E, N, -1)
    offsets = np.concatenate(([0], np.cumsum(sizes))).astype(np.int32)
    out, ok = guarded(torch, (R_, N), dtypes(torch)[kind])
    out.fill_(7.0)
    ta, tsa, tb, tsb, toff = dev(torch, a, sa, b, sb, offsets)
    trows = None if rows is None else dev(torch, np.asarray(rows, np.int32))[0]
    L.lpgemm_mxfp4_grouped(ta, tsa, tb, tsb, toff, rows=trows, out=out)
    assert ok()
    va, vb = R.values(a, sa), R.values(b, sb)
    at = np.arange(R_) if rows is None else np.asarray(rows)
    x = np.where(((at >= 0) & (at < T))[:, None], va[at.clip(0, T - 1)] if T else np.zeros((R_, va.shape[1])), 0.0)
    for e in range(E):
        i, j = offsets[e], offsets[e + 1]
        if j > i:
            held(out[i:j], x[i:j], vb[e], kind, f"group {e}")
    return out


SPLITS = {"one": [40], "even": [16] * 5, "single rows": [1] * 33, "empty ones": [0, 5, 0, 0, 33, 1, 0], "all empty": [0, 0, 0],
          "skewed": [300, 1, 0, 7, 64, 2], "tile edges": [31, 32, 33, 127, 128, 129, 255, 256, 257], "many": [3, 0, 1, 9] * 32,
          "one large": [0, 0, 700, 0]}


@pytest.mark.parametrize("kind", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("split", list(SPLITS))
@pytest.mark.parametrize("N,K", [(96, 512), (301, 2897), (8, 40)])
def test_grouped(torch, kind, split, N, K):
    run_grouped(torch, np.random.default_rng(N), SPLITS[split], N, K, kind)


@pytest.mark.parametrize("split", ["single rows", "empty ones", "skewed", "tile edges", "many"])
def test_grouped_gathered_rows(torch, split):
    """Rows taken through an index, some of them many times, some outside A (zeros)."""
    rng = np.random.default_rng(8)
    n = int(np.sum(SPLITS[split]))
    rows = rng.integers(0, 50, n)
    rows[::7] = -1
    rows[3::11] = 50
    rows[5::13] = 2 ** 31 - 1
    rows[6::17] = -2 ** 31
    out = run_grouped(torch, rng, SPLITS[split], 200, 700, "float32", T=50, rows=rows)
    assert not out[::7].any()


def test_grouped_no_rows_of_a(torch):
    out = run_grouped(torch, np.random.default_rng(0), [3, 2], 64, 256, "float32", T=0, rows=[0, 1, -1, 5, 0])
    assert not out.any()


def test_grouped_rows_in_no_group_stay(torch):
    rng = np.random.default_rng(4)
    a, sa, = R.random_operand(rng, 60, 256)
    b, sb = R.random_operand(rng, 3 * 40, 256)
    b, sb = b.reshape(3, 40, -1), sb.reshape(3, 40, -1)
    va, vb = R.values(a, sa), R.values(b, sb)
    t = dev(torch, a, sa, b, sb)
    for offsets, groups in (([5, 20, 20, 50], [(5, 20), None, (20, 50)]), ([-7, 10, 30, 99], [(0, 10), (10, 30), (30, 60)]),
                            ([0, 40, 20, 20], [(0, 40), None, None]), ([70, 80, 90, 100], [None] * 3),
                            ([-2 ** 31, 2 ** 31 - 1, 0, 0], [(0, 60), None, None])):
        out, ok = guarded(torch, (60, 40), torch.float32)
        out.fill_(7.0)
        L.lpgemm_mxfp4_grouped(*t, dev(torch, np.array(offsets, np.int32))[0], out=out)
        assert ok()
        left = np.ones(60, bool)
        for e, g in enumerate(groups):
            if g:
                held(out[g[0]:g[1]], va[g[0]:g[1]], vb[e], "float32")
                left[g[0]:g[1]] = False
        assert (out.cpu().numpy()[left] == 7.0).all()


def test_grouped_same_as_the_product(torch):
    """One group of all rows has the product's results, to their common bound."""
    rng = np.random.default_rng(2)
    a, sa = R.random_operand(rng, 150, 1000)
    b, sb = R.random_operand(rng, 333, 1000)
    t = dev(torch, a, sa, b, sb)
    one = dev(torch, np.array([0, 150], np.int32))[0]
    held(L.lpgemm_mxfp4_grouped(t[0], t[1], t[2][None], t[3][None], one, dtype=torch.float32), R.values(a, sa), R.values(b, sb), "float32")


# ---- streams and graphs ------------------------------------------------------------
def chain(torch, x, w, sw, offsets, rows):
    codes, scales = L.lpgemm_mxfp4_quantize(x)
    y = L.lpgemm_mxfp4_grouped(codes, scales, w, sw, offsets, rows=rows, dtype=torch.float32)
    z = L.lpgemm_mxfp4(codes, scales, w[0], sw[0], dtype=torch.float32)
    return y, z, L.lpgemm_mxfp4_dequantize(codes, scales, x.shape[1])


@pytest.fixture(params=[(24, 1024), (300, 640), (2, 8192)])
def chained(torch, request):
    T, K = request.param
    rng = np.random.default_rng(T)
    w, sw = R.random_operand(rng, 4 * 96, K)
    w, sw = dev(torch, w.reshape(4, 96, -1), sw.reshape(4, 96, -1))
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
    codes, scales = L.lpgemm_mxfp4_quantize(x, stream=s)
    y = L.lpgemm_mxfp4_grouped(codes, scales, w, sw, offsets, rows=rows, dtype=torch.float32, stream=s)
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
