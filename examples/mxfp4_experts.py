"""A feed-forward layer of routed experts on microscaled 4-bit weights.

    python examples/mxfp4_experts.py [tokens]

Weights are quantised once, as when a model is loaded.  A step quantises the
tokens' hidden states, multiplies each expert's rows with its up projection,
applies the activation, quantises again, multiplies with the down projection
and adds a token's experts up; a shared expert takes every token through the
plain product.  The result is set against the same layer in float32.
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


def route(x, router):
    """(rows, offsets, weights, token): the tokens of every expert in turn."""
    weight, chosen = (x.float() @ router.t()).softmax(1).topk(TOP, 1)
    order = chosen.flatten().argsort(stable=True)
    sizes = torch.bincount(chosen.flatten(), minlength=EXPERTS)
    offsets = torch.cat((sizes.new_zeros(1), sizes.cumsum(0))).int()
    token = order // TOP
    return token.int(), offsets, weight.flatten()[order], token


def layer(x, router, up, down, shared):
    rows, offsets, weight, token = route(x, router)
    a, sa = L.lpgemm_mxfp4_quantize(x)
    h = L.lpgemm_mxfp4_grouped(a, sa, *up, offsets, rows=rows)  # [tokens * TOP, INNER]
    h = torch.nn.functional.silu(h)
    y = L.lpgemm_mxfp4_grouped(*L.lpgemm_mxfp4_quantize(h), *down, offsets, dtype=torch.float32)
    out = L.lpgemm_mxfp4(a, sa, *shared, dtype=torch.float32)
    return out.index_add_(0, token, y * weight[:, None])


def plain(x, router, up, down, shared):
    """The same layer on float32 weights."""
    rows, offsets, weight, token = route(x, router)
    x = x.float()
    out, at = x @ shared.t(), offsets.tolist()
    for e in range(EXPERTS):
        i = slice(at[e], at[e + 1])
        h = torch.nn.functional.silu(x[token[i]] @ up[e].t())
        out.index_add_(0, token[i], (h @ down[e].t()) * weight[i, None])
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
