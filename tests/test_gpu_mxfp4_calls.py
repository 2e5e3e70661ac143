"""The microscaled calls around the kernels: refusals of device tensors, the
native way against the long one, shapes that AUTO picks, sizes past 32 bits
and the example (needs an MI355X)."""
import os
import runpy

import numpy as np
import pytest

import mxfp4_reference as R
import precision_integer_gemm_amd as L
from test_gpu_mxfp4 import dev, dtypes, guarded, held, run_grouped, torch  # noqa: F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def operands(torch):  # noqa: F811
    rng = np.random.default_rng(0)
    a, b = R.random_operand(rng, 6, 300), R.random_operand(rng, 3 * 40, 300)
    b3 = [x.reshape(3, 40, -1) for x in b]
    return dict(zip(("a", "sa", "b", "sb"), dev(torch, *a, *b))), dict(zip(("b", "sb"), dev(torch, *b3)))


def test_refusals_on_the_device(torch, operands):  # noqa: F811
    o, g = operands
    a, sa, b, sb = o.values()
    off = torch.tensor([0, 2, 2, 6], dtype=torch.int32, device="cuda")
    for bad in ((a[:, :128], sa, b, sb), (a, sa[:, :8], b, sb), (a, sa, b[:, :64].contiguous(), sb[:, :4].contiguous()), (a.cpu(), sa, b, sb),
                (a, sa.cpu(), b, sb), (a[None], sa[None], b, sb), (a, sa[:5], b, sb)):
        with pytest.raises(ValueError):
            L.lpgemm_mxfp4(*bad)
    for bad in ((a.int(), sa, b, sb), (a, sa.float(), b, sb), (None, sa, b, sb)):
        with pytest.raises((TypeError, ValueError)):
            L.lpgemm_mxfp4(*bad)
    with pytest.raises(TypeError):
        L.lpgemm_mxfp4(a, sa, b, sb, dtype=torch.float64)
    with pytest.raises(ValueError):
        L.lpgemm_mxfp4(a, sa, b, sb, out=torch.empty(6, 119, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises((TypeError, ValueError)):
        L.lpgemm_mxfp4(a, sa, b, sb, workspace="none")
    for bad, err in (((off[:3],), ValueError), ((off.long(),), TypeError), ((off.cpu(),), ValueError), ((off[None],), ValueError)):
        with pytest.raises(err):
            L.lpgemm_mxfp4_grouped(a, sa, g["b"], g["sb"], *bad)
    with pytest.raises(TypeError):
        L.lpgemm_mxfp4_grouped(a, sa, g["b"], g["sb"], off, rows=off.long())
    with pytest.raises(ValueError):
        L.lpgemm_mxfp4_grouped(a, sa, b, sb, off)
    for K in (-1, 128, 385):
        with pytest.raises(ValueError):
            L.lpgemm_mxfp4_dequantize(a, sa, K)
    x = torch.zeros(4, 64, device="cuda")
    for bad in (x.t(), x[None], x[:, ::2], x.cpu()):
        with pytest.raises(ValueError):
            L.lpgemm_mxfp4_quantize(bad)
    with pytest.raises(TypeError):
        L.lpgemm_mxfp4_quantize(x.double())
    with pytest.raises(ValueError):
        L.lpgemm_mxfp4_quantize(x, codes=torch.empty(4, 63, dtype=torch.uint8, device="cuda"))


def test_the_long_way_gives_the_same(torch, operands):  # noqa: F811
    o, g = operands
    a, sa, b, sb = o.values()
    off = torch.tensor([0, 2, 2, 6], dtype=torch.int32, device="cuda")
    rows = torch.tensor([5, 0, 1, 1, -1, 3], dtype=torch.int32, device="cuda")
    stream = torch.cuda.current_stream()
    for kind in dtypes(torch).values():
        out = torch.empty(6, 120, dtype=kind, device="cuda")
        assert torch.equal(L.lpgemm_mxfp4(a, sa, b, sb, out=out), L.lpgemm_mxfp4(a, sa, b, sb, dtype=kind))
        assert torch.equal(L.lpgemm_mxfp4_grouped(a, sa, g["b"], g["sb"], off, rows=rows, dtype=kind, stream=stream),
                           L.lpgemm_mxfp4_grouped(a, sa, g["b"], g["sb"], off, rows=rows, dtype=kind))
        x = torch.randn(7, 500, device="cuda").to(kind)
        for p, q in zip(L.lpgemm_mxfp4_quantize(x), L.lpgemm_mxfp4_quantize(x, stream=stream)):
            assert torch.equal(p, q)
        assert torch.equal(L.lpgemm_mxfp4_dequantize(a, sa, 300, dtype=kind), L.lpgemm_mxfp4_dequantize(a, sa, 300, dtype=kind, stream=stream))
    class Sub(torch.Tensor):  # not a plain tensor: the long way
        pass
    assert torch.equal(L.lpgemm_mxfp4(a.as_subclass(Sub), sa, b, sb).as_subclass(torch.Tensor), L.lpgemm_mxfp4(a, sa, b, sb))


# each shape that the cost picks, and where it goes over to the next
AUTO = [(513, 6086, 325), (1202, 4895, 35), (300, 4000, 700), (1025, 1023, 4096), (199, 2100, 6277), (250, 8193, 513), (2848, 2873, 200),
        (2100, 4100, 1100), (3000, 300, 128), (4100, 4097, 512), (33, 2000, 9000), (130, 70, 16384), (130, 70, 16500)]


@pytest.mark.parametrize("kind", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("M,N,K", AUTO)
def test_auto(torch, kind, M, N, K):  # noqa: F811
    rng = np.random.default_rng(M + N + K)
    a, sa = R.random_operand(rng, M, K)
    b, sb = R.random_operand(rng, N, K, center=117)
    out, ok = guarded(torch, (M, N), dtypes(torch)[kind])
    L.lpgemm_mxfp4(*dev(torch, a, sa, b, sb), out=out)
    assert ok()
    # some rows of all columns, all rows of some columns
    r, c = np.unique(np.r_[0:3, M - 3:M, rng.integers(0, M, 60)]), np.unique(np.r_[0:3, N - 3:N, rng.integers(0, N, 60)])
    va, vb = R.values(a, sa), R.values(b, sb)
    held(out[torch.from_numpy(r).cuda()], va[r], vb, kind, "rows")
    held(out[:, torch.from_numpy(c).cuda()], va, vb[c], kind, "columns")


@pytest.mark.parametrize("sizes,N,K", [([90] * 12, 1001, 300), ([700, 0, 1200, 3], 1300, 640), ([20] * 100, 300, 400), ([64, 65, 128, 129] * 20, 520, 900),
                                       ([1500, 1, 2600], 2000, 1100)])
def test_auto_grouped(torch, sizes, N, K):  # noqa: F811
    run_grouped(torch, np.random.default_rng(N), sizes, N, K, "bfloat16")


def test_result_past_32_bits(torch):  # noqa: F811
    """2^31 elements and more: the last rows are those of a product of their own."""
    M, N, K = 66000, 33000, 64
    g = torch.Generator("cuda").manual_seed(0)
    u8 = lambda *s: torch.randint(0, 256, s, dtype=torch.uint8, device="cuda", generator=g)  # noqa: E731
    a, b = u8(M, 64), u8(N, 64)
    a[:, 32:], b[:, 32:] = 0, 0
    sa, sb = torch.full((M, 4), 124, dtype=torch.uint8, device="cuda"), torch.full((N, 4), 121, dtype=torch.uint8, device="cuda")
    d = L.lpgemm_mxfp4(a, sa, b, sb)
    for at in (0, 65000, M - 300):
        want = L.lpgemm_mxfp4(a[at:at + 300].contiguous(), sa[at:at + 300].contiguous(), b, sb)
        held(d[at:at + 300, :50], R.values(a[at:at + 300].cpu().numpy(), sa[at:at + 300].cpu().numpy()), R.values(b[:50].cpu().numpy(), sb[:50].cpu().numpy()),
             "bfloat16")
        assert torch.equal(d[at:at + 300], want)  # one group of eight k and one sum: no order to differ in


@pytest.mark.parametrize("rows", [30, 3000])
def test_weights_past_32_bits(torch, rows):  # noqa: F811
    """Matrices of more than 2^32 bytes together: the last expert's rows."""
    E, N, K = 40, 16384, 16384
    b = torch.randint(0, 256, (E, N, K // 2), dtype=torch.uint8, device="cuda")
    sb = torch.randint(115, 121, (E, N, K // 32), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(1)
    a, sa = R.random_operand(rng, rows, K)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = rows
    off[-2] = rows // 3
    ta, tsa = dev(torch, a, sa)
    d = L.lpgemm_mxfp4_grouped(ta, tsa, b, sb, off, dtype=torch.float32)
    cols = [0, 1, 5000, N - 1]
    for e, i in ((E - 2, 0), (E - 1, rows - 1), (E - 1, rows // 3)):
        held(d[i:i + 1, cols], R.values(a, sa)[i:i + 1], R.values(b[e][cols].cpu().numpy(), sb[e][cols].cpu().numpy()), "float32")


def test_quantise_past_32_bits(torch):  # noqa: F811
    rows, K = 70000, 32768
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    x[-50:] = torch.randn(50, K, device="cuda").to(torch.bfloat16)
    codes, scales = L.lpgemm_mxfp4_quantize(x)
    c, s = L.lpgemm_mxfp4_quantize(x[-50:].contiguous())
    assert torch.equal(codes[-50:], c) and torch.equal(scales[-50:], s) and not codes[:-50].any()
    y = L.lpgemm_mxfp4_dequantize(codes, scales, K)
    assert torch.equal(y[-50:], L.lpgemm_mxfp4_dequantize(c, s, K)) and not y[:-50].any()


def test_example(torch, capsys):  # noqa: F811
    runpy.run_path(os.path.join(ROOT, "examples", "mxfp4_experts.py"))["main"](40)
    assert "relative error" in capsys.readouterr().out
