"""Refusals of the routing entry points, on the host before any HIP call (no GPU
needed), and the reference's own checks."""
import ctypes
import math

import numpy as np
import pytest
import torch

import precision_integer_gemm_amd as L
import routing_reference as R
from precision_integer_gemm_amd._binding import RouteOptions

P = 4096
BAD, UNS = L.ERR_INVALID_ARG, L.ERR_UNSUPPORTED
OPTIONS = dict(score=0, top=2, groups=2, top_groups=1, group_top=2, renormalise=1, scale=1.0)
ROUTE = dict(logits=P, dtype=L.OUT_BF16, ldl=8, bias=None, options=OPTIONS, experts=P, weights=P, rows=P, offsets=P, places=P, T=4, E=8, workspace=None, bytes=0)
BACK = dict(dweights=P, logits=P, dtype=L.OUT_F32, ldl=8, experts=P, options=OPTIONS, dlogits=P, T=4, E=8)
COMBINE = dict(y=P, y_dtype=L.OUT_BF16, R=9, places=P, weights=P, residual=P, out=P, dtype=L.OUT_BF16, T=4, top=2, N=16)
COMBINE_BACK = dict(dout=P, dtype=L.OUT_BF16, y=P, y_dtype=L.OUT_BF16, R=9, places=P, weights=P, dy=P, dweights=P, T=4, top=2, N=16)
OPTION_ERRORS = [({"score": 2}, BAD), ({"score": -1}, BAD), ({"top": 0}, BAD), ({"top": -3}, BAD), ({"top": 5}, BAD), ({"groups": 0}, BAD), ({"groups": 3}, BAD),
                 ({"top_groups": 0}, BAD), ({"top_groups": 3}, BAD), ({"group_top": 0}, BAD), ({"group_top": 3}, BAD), ({"renormalise": 2}, BAD),
                 ({"top": L.ROUTE_MAX_TOP + 1}, UNS), ({"groups": L.ROUTE_MAX_GROUPS + 1, "top_groups": 1}, UNS)]


def call(fn, args):
    args = dict(args)
    if isinstance(args.get("options"), dict):
        args["options"] = ctypes.byref(RouteOptions(**args["options"]))
    return getattr(L.lib(), fn)(*args.values(), None)


@pytest.mark.parametrize("fn,args", [("lpgemm_route", ROUTE), ("lpgemm_route_backward", BACK)])
@pytest.mark.parametrize("change,want", OPTION_ERRORS)
def test_options(fn, args, change, want):
    assert call(fn, {**args, "options": {**OPTIONS, **change}}) == want


CASES = [
    *[("lpgemm_route", ROUTE, c, w) for c, w in [
        ({"T": -1}, BAD), ({"E": -1}, BAD), ({"E": 0}, BAD), ({"E": 7}, BAD), ({"dtype": L.OUT_FP8_E4M3}, BAD), ({"ldl": 7}, BAD), ({"ldl": -8}, BAD),
        ({"ldl": 2 ** 61}, BAD), ({"options": None}, BAD), ({"logits": None}, BAD), ({"logits": P + 1}, BAD), ({"bias": P + 2}, BAD), ({"experts": None}, BAD),
        ({"weights": None}, BAD), ({"rows": None}, BAD), ({"offsets": None}, BAD), ({"places": None}, BAD), ({"places": P + 1}, BAD), ({"T": 100}, BAD),
        ({"T": 100, "workspace": P, "bytes": 2}, BAD), ({"T": 100, "workspace": P + 2, "bytes": 4096}, BAD), ({"E": L.ROUTE_MAX_EXPERTS + 2}, UNS),
        ({"T": 2 ** 31}, UNS), ({"T": 2 ** 62}, UNS)]],
    *[("lpgemm_route_backward", BACK, c, w) for c, w in [
        ({"T": -1}, BAD), ({"dtype": 9}, BAD), ({"ldl": 7}, BAD), ({"dweights": None}, BAD), ({"logits": None}, BAD), ({"experts": None}, BAD),
        ({"dlogits": None}, BAD), ({"dlogits": P + 2}, BAD), ({"E": L.ROUTE_MAX_EXPERTS + 2}, UNS)]],
    *[("lpgemm_combine", COMBINE, c, w) for c, w in [
        ({"R": -1}, BAD), ({"T": -1}, BAD), ({"top": -1}, BAD), ({"N": -1}, BAD), ({"y_dtype": 7}, BAD), ({"dtype": L.OUT_FP8_E5M2}, BAD), ({"y": None}, BAD),
        ({"places": None}, BAD), ({"out": None}, BAD), ({"y": P + 1}, BAD), ({"residual": P + 1}, BAD), ({"weights": P + 2}, BAD), ({"out": P + 1}, BAD),
        ({"N": L.COMBINE_MAX_N + 1}, UNS), ({"top": L.COMBINE_MAX_TOP + 1}, UNS), ({"T": 2 ** 31}, UNS), ({"R": 2 ** 31}, UNS)]],
    *[("lpgemm_combine_backward", COMBINE_BACK, c, w) for c, w in [
        ({"R": -1}, BAD), ({"N": -1}, BAD), ({"dtype": 7}, BAD), ({"y_dtype": 8}, BAD), ({"dout": None}, BAD), ({"y": None}, BAD), ({"dy": None}, BAD),
        ({"dweights": None}, BAD), ({"places": None}, BAD), ({"dy": P + 1}, BAD), ({"top": L.COMBINE_MAX_TOP + 1}, UNS)]],
]


@pytest.mark.parametrize("fn,args,change,want", CASES, ids=[f"{c[0][7:]}-{c[2]}" for c in CASES])
def test_argument_errors(fn, args, change, want):
    assert call(fn, {**args, **change}) == want


@pytest.mark.parametrize("fn,args,change", [
    ("lpgemm_route_backward", BACK, {"T": 0, "dlogits": None}), ("lpgemm_combine", COMBINE, {"T": 0, "out": None}), ("lpgemm_combine", COMBINE, {"N": 0, "y": None}),
    ("lpgemm_combine_backward", COMBINE_BACK, {"T": 0}), ("lpgemm_combine_backward", COMBINE_BACK, {"top": 0, "places": None})])
def test_nothing_to_do(fn, args, change):
    assert call(fn, {**args, **change}) == L.OK


def test_workspace_size():
    assert L.lpgemm_route_workspace_size(0, 64) == L.lpgemm_route_workspace_size(16, 1024) == 0
    assert L.lpgemm_route_workspace_size(17, 64) > 0
    for T in (17, 4096, 4097, 8193, 16385, 10 ** 6, 2 ** 24, 2 ** 30):
        assert 0 < L.lpgemm_route_workspace_size(T, 255) <= 2 * 256 * max(256, 1 + T // 60000)
    f = L.lib().lpgemm_route_workspace_size
    n = ctypes.c_size_t(7)
    assert f(4, 4, None) == BAD and f(-1, 4, ctypes.byref(n)) == BAD and f(4, -1, ctypes.byref(n)) == BAD
    assert f(2 ** 31, 4, ctypes.byref(n)) == UNS and f(4, L.ROUTE_MAX_EXPERTS + 1, ctypes.byref(n)) == UNS and n.value == 0


class TestTensorCalls:
    def test_route(self):
        for bad, what in (([1.0], TypeError), (torch.zeros(2, 8, dtype=torch.float64), TypeError), (torch.zeros(8), ValueError), (torch.zeros(2, 8), ValueError)):
            with pytest.raises(what):
                L.lpgemm_route(bad, 2)
        with pytest.raises(ValueError, match="GPU"):
            L.lpgemm_route(torch.zeros(2, 8), 2)
        with pytest.raises(ValueError, match="GPU"):
            L.lpgemm_route_backward(torch.zeros(2, 2), torch.zeros(2, 8), torch.zeros(2, 2, dtype=torch.int32))

    def test_combine(self):
        y, p = torch.zeros(4, 8), torch.zeros(2, 2, dtype=torch.int32)
        for bad, what in (((y.double(), p), TypeError), ((y[0], p), ValueError), ((y, p), ValueError)):
            with pytest.raises(what):
                L.lpgemm_combine(*bad)
            with pytest.raises(what):
                L.lpgemm_combine_backward(torch.zeros(2, 8), *bad)


class TestReference:
    """The reference against PyTorch where that has the operation."""

    def test_softmax_top(self):
        x = torch.randn(20, 16, dtype=torch.float64)
        experts, weights, rows, offsets, places = R.route(x.numpy(), 4)
        want = torch.softmax(x, 1).topk(4, 1)
        np.testing.assert_array_equal(experts, want.indices.numpy())
        np.testing.assert_allclose(weights, (want.values / want.values.sum(1, keepdim=True)).numpy(), rtol=1e-12)
        for t in range(20):
            for k in range(4):
                i = places[t, k]
                assert rows[i] == t and offsets[experts[t, k]] <= i < offsets[experts[t, k] + 1]

    @pytest.mark.parametrize("score", ["softmax", "sigmoid"])
    @pytest.mark.parametrize("renormalise", [True, False])
    def test_gradient_is_autograd_s(self, score, renormalise):
        x, dw = torch.randn(6, 10, dtype=torch.float64, requires_grad=True), torch.randn(6, 3, dtype=torch.float64)
        experts = R.route(x.detach().numpy(), 3, score)[0]
        p = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
        w = p.gather(1, torch.from_numpy(experts).long())
        w = w / w.sum(1, keepdim=True) if renormalise else w
        (1.5 * w * dw).sum().backward()
        np.testing.assert_allclose(R.route_gradient(dw.numpy(), x.detach().numpy(), experts, score, renormalise, 1.5), x.grad.numpy(), atol=1e-12)

    def test_groups_and_masks(self):
        x = np.array([[3.0, 1, 2.9, 2.8, -math.inf, 5, 0, 0]])
        assert R.route(x, 3, "sigmoid", groups=4, top_groups=2, group_top=1)[0].tolist() == [[5, 0, 1]]
        # sums of sigmoids: 0.953 + 0.731, 0.948 + 0.943, 0.993 alone, 0.5 + 0.5
        assert R.route(x, 3, "sigmoid", groups=4, top_groups=2, group_top=2)[0].tolist() == [[0, 2, 3]]
        assert R.route(np.full((1, 4), -math.inf), 2)[0].tolist() == [[-1, -1]]
        assert R.route(np.array([[1.0, 1, 1, 1]]), 2)[0].tolist() == [[0, 1]]


@pytest.mark.parametrize("name", ["top", "groups", "top_groups", "group_top"])
@pytest.mark.parametrize("value", [2 ** 32 + 1, -2 ** 32 + 1, 2 ** 31])
def test_sizes_past_the_options_fields(name, value):
    from precision_integer_gemm_amd import _binding
    given = {"top": 2, "score": "softmax", "groups": 4, "top_groups": 1, "group_top": 1, "renormalise": True, "scale": 1.0}
    made = _binding._route_options(**given)
    assert (made.top, made.groups, made.top_groups, made.group_top) == (2, 4, 1, 1)
    with pytest.raises(ValueError, match=name):
        _binding._route_options(**{**given, name: value})
