"""A feed-forward layer of routed experts on microscaled 4-bit weights.

    python examples/mxfp4_experts.py [tokens]

Weights are quantised once, as when a model is loaded.  A step routes the tokens,
quantises their hidden states, multiplies each expert's rows with its up
projection, applies the activation, quantises again, multiplies with the down
projection and adds a token's experts up; a shared expert takes every token through
the plain product.  The result is set against the same layer in float32.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import precision_integer_gemm_amd as L  # noqa: E402

HIDDEN, INNER, EXPERTS, TOP = 1024, 2048, 16, 4


def quantised(w):
    """Codes and scales of weights [..., N, K]."""
    codes, scales = L.lpgemm_mxfp4_quantize(w.flatten(0, -2))
    return codes.view(*w.shape[:-1], -1), scales.view(*w.shape[:-1], -1)


def layer(x, router, up, down, shared):
    r = L.lpgemm_route(x.float() @ router.t(), TOP, renormalise=False)
    a, sa = L.lpgemm_mxfp4_quantize(x)
    h = L.lpgemm_mxfp4_grouped(a, sa, *up, r.offsets, rows=r.rows)  # [tokens * TOP, INNER]
    h = torch.nn.functional.silu(h)
    y = L.lpgemm_mxfp4_grouped(*L.lpgemm_mxfp4_quantize(h), *down, r.offsets, dtype=torch.float32)
    out = L.lpgemm_mxfp4(a, sa, *shared, dtype=torch.float32)
    return L.lpgemm_combine(y, r.places, r.weights, residual=out)


def plain(x, router, up, down, shared):
    """The same layer on float32 weights."""
    x = x.float()
    weight, chosen = (x @ router.t()).softmax(1).topk(TOP, 1)
    out = x @ shared.t()
    for e in range(EXPERTS):
        token, k = torch.where(chosen == e)
        h = torch.nn.functional.silu(x[token] @ up[e].t())
        out.index_add_(0, token, (h @ down[e].t()) * weight[token, k, None])
    return out


def main(tokens=64):
    g = torch.Generator("cuda").manual_seed(0)
    w = lambda *s: torch.randn(*s, device="cuda", generator=g) / s[-1] ** 0.5  # noqa: E731
    router, up, down, shared = w(EXPERTS, HIDDEN), w(EXPERTS, INNER, HIDDEN), w(EXPERTS, HIDDEN, INNER), w(HIDDEN, HIDDEN)
    x = torch.randn(tokens, HIDDEN, device="cuda", generator=g).to(torch.bfloat16)
    packed = [quantised(t) for t in (up, down, shared)]
    got = layer(x, router, *packed)
    want = plain(x, router, up, down, shared)
    # weights' and activations' 4 bits: each value is off by up to a quarter of a binade
    error = float((got - want).norm() / want.norm())
    print(f"{tokens} tokens, {EXPERTS} experts, top {TOP}: relative error against float32 weights {error:.3f}")
    assert error < 0.35
    # against the values that the codes stand for, only the second quantisation's input rounding is left
    values = [L.lpgemm_mxfp4_dequantize(c.flatten(0, -2), s.flatten(0, -2), t.shape[-1], dtype=torch.float32).view_as(t)
              for (c, s), t in zip(packed, (up, down, shared))]
    xq = L.lpgemm_mxfp4_dequantize(*L.lpgemm_mxfp4_quantize(x), HIDDEN)
    out = torch.nn.functional.linear(xq.float(), values[2])
    print(f"shared expert against the codes' values: {float((L.lpgemm_mxfp4(*L.lpgemm_mxfp4_quantize(x), *packed[2], dtype=torch.float32) - out).abs().max()):.2e}")


if __name__ == "__main__":
    main(*(int(v) for v in sys.argv[1:2]))
