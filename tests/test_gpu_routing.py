"""Routing to experts, the sum of a token's experts, and both gradients, against
float64 references written from their definitions."""
import math

import numpy as np
import pytest

import precision_integer_gemm_amd as L
import routing_reference as R

pytestmark = pytest.mark.gpu
KINDS = ["float32", "bfloat16", "float16"]
HALF_STEP = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
LEAST = {"float32": 2.0 ** -149, "bfloat16": 2.0 ** -133, "float16": 2.0 ** -24}


@pytest.fixture(scope="module")
def torch():
    import torch
    return torch


def kind_of(torch, kind):
    return getattr(torch, kind)


def check_route(torch, logits, top, bias=None, **how):
    got = L.lpgemm_route(logits, top, bias=bias, **how)
    x = logits.double().cpu().numpy()
    want = R.route(x, top, bias=None if bias is None else bias.cpu().numpy(), **how)
    np.testing.assert_array_equal(got.experts.cpu().numpy(), want[0])
    np.testing.assert_array_equal(got.offsets.cpu().numpy(), want[3])
    np.testing.assert_array_equal(got.rows.cpu().numpy(), want[2])
    np.testing.assert_array_equal(got.places.cpu().numpy(), want[4])
    # binary64 scores: the type's rounding alone.  binary32 ones: exponentials and their argument to 2 steps each, a sum of
    # up to 1024 of them in 16 + 6 steps, a quotient, a product by scale, 32 chosen ones added
    np.testing.assert_allclose(got.weights.cpu().numpy(), want[1], rtol=64 * 2.0 ** -24, atol=1e-37)
    return got


SHAPES = [(1, 1, 1), (1, 256, 8), (3, 8, 2), (16, 32, 4), (17, 64, 8), (65, 60, 6), (129, 128, 8), (200, 100, 16), (70, 384, 8), (33, 512, 32), (20, 1000, 7),
          (5, 1024, 32)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,top", SHAPES)
def test_route(torch, kind, score, T, E, top):
    g = torch.Generator("cuda").manual_seed(T + E)
    x = (2 * torch.randn(T, E, device="cuda", generator=g)).to(kind_of(torch, kind))
    bias = 0.1 * torch.randn(E, device="cuda", generator=g)
    for renormalise in (True, False):
        check_route(torch, x, top, score=score, renormalise=renormalise)
        check_route(torch, x, top, bias, score=score, renormalise=renormalise, scale=2.5)


GROUPED = [(1, 256, 8, 8, 4), (40, 64, 6, 8, 3), (33, 160, 6, 8, 3), (20, 65, 5, 13, 4), (7, 64, 1, 64, 1), (9, 128, 2, 64, 2), (50, 30, 10, 3, 2), (3, 1024, 16, 16, 5),
           (12, 512, 8, 4, 1), (64, 96, 4, 4, 4)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("T,E,top,groups,top_groups", GROUPED)
def test_route_groups(torch, score, group_top, T, E, top, groups, top_groups):
    g = torch.Generator("cuda").manual_seed(T + E)
    x = 2 * torch.randn(T, E, device="cuda", generator=g)
    x[torch.rand(T, E, device="cuda", generator=g) < 0.1] = -math.inf
    bias = 0.1 * torch.randn(E, device="cuda", generator=g)
    how = dict(score=score, groups=groups, top_groups=top_groups, group_top=group_top)
    check_route(torch, x, top, **how)
    check_route(torch, x, top, bias, **how)
    check_route(torch, x.half(), top, bias, **how)


@pytest.mark.parametrize("T,top", [(4095, 1), (4096, 2), (4097, 1), (5000, 3), (16385, 1), (20000, 2)])
def test_route_lists_of_many_tokens(torch, T, top):
    """Workgroups, rounds and stretches of every kind: the lists of the experts that were chosen."""
    E = 13
    x = torch.randn(T, E, device="cuda", generator=torch.Generator("cuda").manual_seed(T))
    x[::5] = -math.inf
    got = L.lpgemm_route(x, top)
    experts = got.experts.long()
    want = x.sort(dim=1, descending=True, stable=True).indices[:, :top]
    assert torch.equal(experts, torch.where((x[:, :1] == -math.inf), -1, want))
    flat = torch.where(experts < 0, E, experts).flatten()
    order = flat.argsort(stable=True)
    used = int((flat < E).sum())
    assert got.offsets.tolist() == [int((flat < e).sum()) for e in range(E + 1)]
    assert torch.equal(got.rows[:used].long(), order[:used] // top) and (got.rows[used:] == -1).all()
    places = torch.empty_like(flat)
    places[order] = torch.arange(T * top, device="cuda")
    assert torch.equal(got.places.long().flatten(), torch.where(flat < E, places, -1))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("how", [dict(), dict(groups=4, top_groups=2), dict(groups=4, top_groups=2, group_top=1)])
@pytest.mark.parametrize("biased", [False, True])
def test_route_masks(torch, kind, score, how, biased):
    """Closed experts, rows of them, the type's lowest value, equal logits, zeros of both signs."""
    dtype = kind_of(torch, kind)
    low = torch.finfo(dtype).min
    x = torch.randn(24, 16, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).to(dtype)
    x[0] = -math.inf
    x[1, 1:] = -math.inf
    x[2, :14] = -math.inf
    x[3] = low
    x[4, 2:] = low
    x[5] = 1.5
    x[6, ::2] = 0.0
    x[6, 1::2] = -0.0
    x[7] = x[7].round()
    x[8, :8] = -math.inf
    x[9, 4:] = -math.inf
    x[23] = -math.inf
    bias = None
    if biased:
        bias = torch.full((16,), 0.25, device="cuda")
        bias[5:9] = torch.tensor([-0.5, 0.25, -3.4e38, 0.75], device="cuda")
    got = check_route(torch, x, 4, bias, score=score, **how)
    assert (got.experts[0] == -1).all() and (got.weights[0] == 0).all() and not got.weights.isnan().any()
    check_route(torch, x, 4, bias, score=score, renormalise=False, **how)


@pytest.mark.parametrize("biased", [False, True])
def test_route_nan_ranks_first(torch, biased):
    x = torch.randn(6, 20, device="cuda")
    x[1, 7], x[2, 19], x[2, 3], x[3, 0] = math.nan, math.nan, math.nan, math.inf
    bias = torch.zeros(20, device="cuda") if biased else None
    got = L.lpgemm_route(x, 3, score="sigmoid", bias=bias, renormalise=False)
    assert got.experts[1, 0] == 7 and got.experts[2, :2].tolist() == [3, 19] and got.experts[3, 0] == 0
    assert got.weights[1, 0].isnan() and not got.weights[1, 1:].isnan().any() and got.weights[3, 0] == 1
    soft = L.lpgemm_route(x, 3, bias=bias)
    assert soft.weights[1:4].isnan().all() and not soft.weights[[0, 4, 5]].isnan().any()
    assert ((soft.experts >= 0) & (soft.experts < 20)).all()


def test_route_neighbours_next_to_a_border(torch):
    """Choice scores that binary32 takes for equal still order."""
    x = torch.zeros(2, 64, device="cuda")
    x[0, 40] = 1e-6  # sigmoid differs by 2.5e-7 ...
    bias = torch.full((64,), 16.0, device="cuda")  # ... which is below half a step of binary32 at 16
    check_route(torch, x, 2, bias, score="sigmoid")
    x[1, 40] = -1e-6
    got = check_route(torch, x, 2, bias, score="sigmoid")
    assert got.experts[0].tolist() == [40, 0] and got.experts[1].tolist() == [0, 1]


def test_route_strided_and_empty(torch):
    x = torch.randn(50, 100, device="cuda")
    check_route(torch, x[:, 3:67], 4)
    check_route(torch, x[::2, 1:8], 3, score="sigmoid")
    check_route(torch, x[:1, 50:], 3)
    got = L.lpgemm_route(x[:0], 4)
    assert got.offsets.tolist() == [0] * 101 and got.experts.shape == (0, 4)


# ---- the logits' gradient --------------------------------------------------------------
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("T,E,top", [(1, 2, 2), (5, 8, 2), (30, 64, 8), (9, 100, 4), (13, 256, 8), (6, 400, 16), (3, 1024, 32)])
def test_route_gradient(torch, kind, score, renormalise, T, E, top):
    g = torch.Generator("cuda").manual_seed(T + E)
    x = (2 * torch.randn(T, E, device="cuda", generator=g)).to(kind_of(torch, kind))
    x[T // 2, 1:] = -math.inf
    dw = torch.randn(T, top, device="cuda", generator=g)
    r = L.lpgemm_route(x, top, score=score, renormalise=renormalise, scale=1.5)
    got = L.lpgemm_route_backward(dw, x, r.experts, score=score, renormalise=renormalise, scale=1.5).double().cpu().numpy()
    experts = r.experts.cpu().numpy()
    want = R.route_gradient(dw.cpu().numpy(), x.double().cpu().numpy(), experts, score, renormalise, 1.5)
    # the terms that are subtracted, each of a few dozen binary32 steps
    p = np.stack([R.scores(v, score) for v in x.double().cpu().numpy()])
    S = np.stack([p[t][experts[t][experts[t] >= 0]].sum() for t in range(T)])[:, None] if renormalise else 1.0
    size = 1.5 * p * 2 * np.abs(dw.cpu().numpy()).max(1, keepdims=True) / S
    off = np.abs(got - want)
    assert (off <= 64 * 2.0 ** -24 * size + HALF_STEP[kind] * np.abs(want) + LEAST[kind]).all(), (off / (size + 1e-30)).max()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
def test_route_gradient_by_differences(torch, score, renormalise):
    """Against differences of the weights themselves, the experts held."""
    T, E, top, h = 4, 12, 3, 1e-5
    rng = np.random.default_rng(0)
    x, dw = rng.standard_normal((T, E)).astype(np.float32), rng.standard_normal((T, top)).astype(np.float32)
    experts = R.route(x, top, score)[0]

    def loss(v):
        total = 0.0
        for t in range(T):
            p = R.scores(v[t], score)[experts[t]]
            total += float((dw[t] * (p / p.sum() if renormalise else p)).sum())
        return total
    want = np.zeros((T, E))
    for t in range(T):
        for e in range(E):
            up, down = x.astype(np.float64), x.astype(np.float64)
            up[t, e] += h
            down[t, e] -= h
            want[t, e] = (loss(up) - loss(down)) / (2 * h)
    got = L.lpgemm_route_backward(*(torch.from_numpy(a).cuda() for a in (dw, x, experts)), score=score, renormalise=renormalise)
    # differences: h^2 of third derivatives below 10, and 1e-16 of sums below 10 over 2 h
    np.testing.assert_allclose(got.cpu().numpy(), want, atol=1e-8 + 64 * 2.0 ** -24 * 10)


# ---- combine -------------------------------------------------------------------------------
def some_places(rng, T, top, R_, none=0.2):
    places = rng.permutation(max(T * top, R_))[:T * top].reshape(T, top).astype(np.int32)
    places[places >= R_] = -1
    places[rng.random((T, top)) < none] = -1
    return places


COMBINE = [(1, 1, 1, 1), (1, 4, 4, 4096), (16, 4, 64, 1000), (3, 2, 9, 7), (40, 8, 320, 129), (5, 32, 160, 333), (300, 2, 500, 2049), (2, 9, 18, 5000), (7, 0, 3, 16)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,top,R_,N", COMBINE)
def test_combine(torch, kind, T, top, R_, N):
    rng = np.random.default_rng(T + N)
    dtype = kind_of(torch, kind)
    y = torch.from_numpy(rng.standard_normal((R_, N))).to(dtype).cuda()
    places, w = some_places(rng, T, top, R_), rng.standard_normal((T, top)).astype(np.float32)
    if T > 2 and top > 1:
        places[1] = places[0, 0]  # the same row several times
        places[2] = R_
    residual = torch.from_numpy(rng.standard_normal((T, N))).to(dtype).cuda()
    tp, tw = torch.from_numpy(places).cuda(), torch.from_numpy(w).cuda()
    for weights, res in ((tw, None), (None, residual), (tw, residual)):
        for out_kind in {kind, "float32"}:
            r = None if res is None else res.to(kind_of(torch, out_kind))
            buffer = torch.full((T * N + 128,), 3.0, dtype=kind_of(torch, out_kind), device="cuda")
            out = buffer[64:64 + T * N].view(T, N)
            L.lpgemm_combine(y, tp, weights, residual=r, out=out)
            assert (buffer[:64] == 3).all() and (buffer[64 + T * N:] == 3).all()
            want, size = R.combine(y.double().cpu().numpy(), places, None if weights is None else w, None if r is None else r.double().cpu().numpy())
            off = np.abs(out.double().cpu().numpy() - want)
            step = 1.01 * (top + 1) * 2.0 ** -24 * size
            assert (off <= step + HALF_STEP[out_kind] * (np.abs(want) + step) + LEAST[out_kind]).all()


def test_combine_in_place_and_padding(torch):
    y = torch.full((4, 100), math.nan, device="cuda")
    y[1] = 2.0
    residual = torch.randn(3, 100, device="cuda")
    places = torch.tensor([[1, -1], [-1, 4], [1, 1]], dtype=torch.int32, device="cuda")
    weights = torch.tensor([[0.5, math.nan], [math.inf, 1.0], [1.0, 2.0]], device="cuda")
    want = residual + torch.tensor([[1.0], [0.0], [6.0]], device="cuda")
    assert torch.equal(L.lpgemm_combine(y, places, weights, residual=residual, out=residual), want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,top,R_,N", COMBINE)
def test_combine_gradient(torch, kind, T, top, R_, N):
    rng = np.random.default_rng(T + N)
    dtype = kind_of(torch, kind)
    y, d = (torch.from_numpy(rng.standard_normal(s)).to(dtype).cuda() for s in ((R_, N), (T, N)))
    places, w = some_places(rng, T, top, R_), rng.standard_normal((T, top)).astype(np.float32)
    buffer = torch.full((R_ * N + 128,), 3.0, dtype=dtype, device="cuda")
    dy = buffer[64:64 + R_ * N].view(R_, N)
    got, dw = L.lpgemm_combine_backward(d, y, torch.from_numpy(places).cuda(), torch.from_numpy(w).cuda(), dy=dy)
    assert got is dy and (buffer[:64] == 3).all() and (buffer[64 + R_ * N:] == 3).all()
    yv, dv, dy, dw = (t.double().cpu().numpy() for t in (y, d, dy, dw))
    left = np.ones(R_, bool)
    for t in range(T):
        for k in range(top):
            i = places[t, k]
            if i < 0:
                assert dw[t, k] == 0
                continue
            left[i] = False
            v = float(w[t, k]) * dv[t]
            assert (np.abs(dy[i] - v) <= (2.0 ** -24 + HALF_STEP[kind]) * 1.001 * np.abs(v) + LEAST[kind]).all()
            # up to N / 2048 terms a lane and column, 8 columns, 64 lanes, 4 waves
            steps = -(-N // 2048) * 8 + 6 + 3
            assert abs(dw[t, k] - (dv[t] * yv[i]).sum()) <= 1.01 * steps * 2.0 ** -24 * np.abs(dv[t] * yv[i]).sum()
    assert (dy[left] == 3).all()


# ---- together, on streams and in graphs ----------------------------------------------------------
HIDDEN, INNER, EXPERTS, TOP = 256, 384, 8, 3


def layer_weights(torch):
    g = torch.Generator("cuda").manual_seed(1)
    w = lambda *s: torch.randn(*s, device="cuda", generator=g) / s[-1] ** 0.5  # noqa: E731
    router, up, down = w(EXPERTS, HIDDEN), w(EXPERTS, INNER, HIDDEN), w(EXPERTS, HIDDEN, INNER)
    bias = 0.05 * torch.randn(EXPERTS, device="cuda", generator=g)

    def quantised(t):
        made = [L.lpgemm_fp8_block_quantize(m, block_rows=128) for m in t]
        return torch.stack([c for c, _ in made]), torch.stack([s for _, s in made])
    return router, bias, quantised(up), quantised(down)


def layer(torch, x, router, bias, up, down):
    """Hidden states to routed experts and back: every operator once."""
    r = L.lpgemm_route(x.float() @ router.t(), TOP, score="sigmoid", bias=bias, groups=4, top_groups=3)
    a, sa = L.lpgemm_fp8_block_quantize(x)
    h = torch.nn.functional.silu(L.lpgemm_fp8_block_grouped(a, sa, *up, r.offsets, rows=r.rows, out=x.new_zeros(len(r.rows), INNER)))
    y = L.lpgemm_fp8_block_grouped(*L.lpgemm_fp8_block_quantize(h), *down, r.offsets, out=x.new_zeros(len(r.rows), HIDDEN))
    return r, L.lpgemm_combine(y, r.places, r.weights, residual=x)


def test_layer_of_experts(torch):
    router, bias, up, down = weights = layer_weights(torch)
    x = torch.randn(90, HIDDEN, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).bfloat16()
    r, got = layer(torch, x, *weights)
    w_up, w_down = (torch.stack([L.lpgemm_fp8_block_dequantize(c, s, c.shape[-1], dtype=torch.float32) for c, s in zip(*w)]) for w in (up, down))
    want = x.float()
    for k in range(TOP):
        e = r.experts[:, k].long()
        h = torch.nn.functional.silu(torch.stack([w_up[e[t]] @ x[t].float() for t in range(90)]))
        want = want + r.weights[:, k:k + 1] * torch.stack([w_down[e[t]] @ h[t] for t in range(90)])
    # two conversions of the activations to three bits of mantissa, each 2^-4 at most and 2^-5.5 on average
    assert float((got.float() - want).norm() / (want - x.float()).norm()) < 0.06


@pytest.mark.parametrize("T", [1, 20, 300])
def test_layer_on_another_stream_and_in_a_graph(torch, T):
    weights = layer_weights(torch)
    x = torch.randn(T, HIDDEN, device="cuda", generator=torch.Generator("cuda").manual_seed(2)).bfloat16()

    def whole(x):
        r, out = layer(torch, x, *weights)
        logits = x.float() @ weights[0].t()
        return [*r, out, L.lpgemm_route_backward(r.weights, logits, r.experts, score="sigmoid")]
    want = whole(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = whole(x)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    static = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = whole(static)
    for seed in range(4):
        new = torch.randn(x.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).bfloat16()
        static.copy_(new)
        graph.replay()
        torch.cuda.synchronize()
        want = whole(new)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), seed


def test_route_same_lists_again(torch):
    x = torch.randn(6000, 64, device="cuda").bfloat16()
    first = L.lpgemm_route(x, 6)
    small = torch.empty(L.lpgemm_route_workspace_size(6000, 64), dtype=torch.uint8, device="cuda")
    for fill in (0, 0x7B, 0xFF):
        small.fill_(fill)
        assert all(torch.equal(a, b) for a, b in zip(L.lpgemm_route(x, 6, workspace=small), first))
    with pytest.raises(L.LpgemmError):
        L.lpgemm_route(x, 6, workspace=small[:-4])
    with pytest.raises(L.LpgemmError):
        L.lpgemm_route(x, 6, workspace=None)
