"""Routing under other circumstances than one call on its own (needs an MI355X):
streams, graphs, random options, and the lists as the grouped products read them."""
import math
import random

import numpy as np
import pytest

import precision_integer_gemm_amd as L
import routing_reference as R
from test_gpu_routing import check_route, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(60))
def test_random_options(torch, seed):  # noqa: F811
    rng = random.Random(seed)
    groups = rng.choice((1, 1, 2, 4, 7, 16, 64))
    E = groups * max(1, round(2 ** rng.uniform(0, 10 - math.log2(groups))))
    E = min(E, 1024 // groups * groups)
    top_groups = rng.randrange(1, groups + 1)
    top = rng.randrange(1, min(32, E // groups * top_groups) + 1)
    T = round(2 ** rng.uniform(0, 8))
    g = torch.Generator("cuda").manual_seed(seed)
    x = rng.choice((0.1, 1.0, 5.0)) * torch.randn(T, E, device="cuda", generator=g)
    x = x.to(rng.choice((torch.float32, torch.bfloat16, torch.float16)))
    if rng.random() < 0.5:
        x[torch.rand(T, E, device="cuda", generator=g) < rng.choice((0.05, 0.9))] = -math.inf
    if rng.random() < 0.3:
        x = x.round()  # many ties
    bias = torch.randn(E, device="cuda", generator=g) * 0.1 if rng.random() < 0.5 else None
    check_route(torch, x, top, bias, score=rng.choice(("softmax", "sigmoid")), groups=groups, top_groups=top_groups, group_top=rng.choice((1, 2)),
                renormalise=rng.random() < 0.5, scale=rng.choice((1.0, 2.5)))


def test_two_streams_at_once(torch):  # noqa: F811
    xs = [torch.randn(5000, 64, device="cuda"), torch.randn(7000, 96, device="cuda").bfloat16()]
    want = [L.lpgemm_route(x, 4) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(L.lpgemm_route(xs[i], 4))
    for i in range(2):
        got[i].append(L.lpgemm_route(xs[i], 4, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


def test_two_graphs(torch):  # noqa: F811
    """Each graph keeps the workspace that it was captured with."""
    xs = [torch.randn(5000, 64, device="cuda") for _ in range(2)]
    graphs, held = [], []
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(L.lpgemm_route(x, 4, score="sigmoid"))
        graphs.append(g)
    for seed in range(3):
        for x in xs:
            x.copy_(torch.randn(x.shape, device="cuda"))
        L.lpgemm_route(xs[0], 8)  # eager work between
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for x, h in zip(xs, held):
            assert all(torch.equal(a, b) for a, b in zip(h, L.lpgemm_route(x, 4, score="sigmoid"))), seed


@pytest.mark.parametrize("T", [1, 16, 17, 300, 9000])
def test_padding_goes_nowhere(torch, T):  # noqa: F811
    """Rows of closed experts at a batch's end: no row is theirs, and the product leaves the rows behind the last one."""
    x = torch.randn(T, 8, device="cuda")
    pad = T // 3
    x[T - pad:] = -math.inf
    r = L.lpgemm_route(x, 2)
    used = 2 * (T - pad)
    assert int(r.offsets[-1]) == used and (r.rows[used:] == -1).all() and (r.places[T - pad:] == -1).all()
    assert torch.equal(r.rows[:used].sort().values, torch.arange(T - pad, device="cuda").int().repeat_interleave(2))
    a, sa = L.lpgemm_fp8_block_quantize(torch.randn(T, 128, device="cuda"))
    b, sb = L.lpgemm_fp8_block_quantize(torch.randn(8 * 128, 128, device="cuda"), block_rows=128)
    out = torch.full((2 * T, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    L.lpgemm_fp8_block_grouped(a, sa, b.view(8, 128, 128), sb.view(8, 1, 1), r.offsets, rows=r.rows, out=out)
    assert (out[used:] == 7).all() and not (out[:used] == 7).all(1).any()
    y = L.lpgemm_combine(out, r.places, r.weights)
    assert not y[T - pad:].any()


def test_the_lists_drive_the_microscaled_product(torch):  # noqa: F811
    x, w = torch.randn(40, 256, device="cuda"), torch.randn(6 * 64, 256, device="cuda")
    r = L.lpgemm_route(torch.randn(40, 6, device="cuda"), 2)
    a, sa = L.lpgemm_mxfp4_quantize(x)
    b, sb = L.lpgemm_mxfp4_quantize(w)
    y = L.lpgemm_mxfp4_grouped(a, sa, b.view(6, 64, -1), sb.view(6, 64, -1), r.offsets, rows=r.rows, dtype=torch.float32)
    got = L.lpgemm_combine(y, r.places, r.weights)
    va, vb = L.lpgemm_mxfp4_dequantize(a, sa, 256, dtype=torch.float32), L.lpgemm_mxfp4_dequantize(b, sb, 256, dtype=torch.float32).view(6, 64, 256)
    for t in range(40):
        want = sum(float(r.weights[t, k]) * (vb[int(r.experts[t, k])] @ va[t]) for k in range(2))
        # binary32 sums of 256 terms on either side
        assert float((got[t] - want).abs().max()) <= 4 * 256 * 2.0 ** -24 * float((vb.abs() @ va[t].abs()).max())


def test_gradient_through_the_layer_s_end(torch):  # noqa: F811
    """combine, its gradients and the router's, against differences of the loss in float64."""
    T, E, top, N, h = 5, 6, 2, 8, 1e-6
    rng = np.random.default_rng(0)
    x, dout = rng.standard_normal((T, E)), rng.standard_normal((T, N))
    experts, _, rows, offsets, places = R.route(x.astype(np.float32), top, "sigmoid")
    y = rng.standard_normal((T * top, N))

    def loss(x):
        w = np.stack([R.scores(x[t], "sigmoid")[experts[t]] for t in range(T)])
        w /= w.sum(1, keepdims=True)
        return float((R.combine(y, places, w)[0] * dout).sum())
    x = x.astype(np.float32).astype(np.float64)
    want = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        d = np.zeros_like(x)
        d[i] = h
        want[i] = (loss(x + d) - loss(x - d)) / (2 * h)
    dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()  # noqa: E731
    logits = dev(x, torch.float32)
    r = L.lpgemm_route(logits, top, score="sigmoid")
    dy, dw = L.lpgemm_combine_backward(dev(dout, torch.float32), dev(y, torch.float32), r.places, r.weights)
    got = L.lpgemm_route_backward(dw, logits, r.experts, score="sigmoid").double().cpu().numpy()
    # values of a few units to 2^-24 through some dozens of steps; differences to 1e-15 / h
    np.testing.assert_allclose(got, want, atol=1e-4)
    np.testing.assert_allclose(dy.double().cpu().numpy()[r.places.cpu().numpy()], r.weights.double().cpu().numpy()[..., None] * dout[:, None], atol=1e-5)
