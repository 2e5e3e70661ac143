"""The microscaled 4-bit operators as a user's program calls them, with plain forms of each.

Three paths: `quantise` takes rows of bf16, fp16 or fp32 values to 4-bit codes
with one power-of-two scale per 32 values and back to the values these stand
for; `product` multiplies two such matrices; `grouped` multiplies the rows
routed to each expert by that expert's matrix.  With `own` false everything is
computed with elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
WIDTH = {"bf16": 2, "f16": 2, "f32": 4}
UNIT = 128  # values of a row per 64 code bytes and 4 scale bytes


def listed():
    return [
        # one token's hidden state on its way into a 4-bit layer: the smallest call, all latency
        {"name": "quantise-token", "op": "quantise", "rows": 1, "K": 8192, "type": "bf16", "stride": 0},
        # a prompt's activations as a slice of a wider buffer: odd length, rows not aligned
        {"name": "quantise-odd-strided", "op": "quantise", "rows": 1001, "K": 2897, "type": "f16", "stride": 2913},
        # fp32 master weights of a square layer, converted when a model is loaded
        {"name": "quantise-weights-f32", "op": "quantise", "rows": 8192, "K": 8192, "type": "f32", "stride": 0},
        # decoding one token through a square layer: the weights are read once, little else happens
        {"name": "product-decode-1", "op": "product", "M": 1, "N": 4096, "K": 4096, "type": "bf16"},
        # decoding a batch of sixteen through an up projection
        {"name": "product-decode-16", "op": "product", "M": 16, "N": 28672, "K": 8192, "type": "bf16"},
        # odd sizes on all sides, results kept in fp32
        {"name": "product-odd-f32", "op": "product", "M": 333, "N": 1001, "K": 2897, "type": "f32"},
        # a prompt through a rectangular layer whose edges end inside tiles
        {"name": "product-prompt-ragged", "op": "product", "M": 3000, "N": 5120, "K": 6144, "type": "f16"},
        # the largest: a long prompt through a square layer
        {"name": "product-prompt-8192", "op": "product", "M": 8192, "N": 8192, "K": 8192, "type": "bf16"},
        # decoding sixteen tokens, four of thirty-two experts each: most experts have a row or two, some none
        {"name": "grouped-decode", "op": "grouped", "T": 16, "top": 4, "E": 32, "N": 4096, "K": 4096, "type": "bf16", "skew": 1.0},
        # a short prompt on many narrow experts: tens of rows each
        {"name": "grouped-short", "op": "grouped", "T": 512, "top": 8, "E": 64, "N": 2048, "K": 4096, "type": "f16", "skew": 0.5},
        # odd sizes, strongly skewed: some experts empty, one with most of the rows
        {"name": "grouped-odd-skewed", "op": "grouped", "T": 555, "top": 2, "E": 13, "N": 1001, "K": 2897, "type": "f32", "skew": 2.0},
        # a long prompt, two of thirty-two experts for each token
        {"name": "grouped-prompt", "op": "grouped", "T": 8192, "top": 2, "E": 32, "N": 4096, "K": 4096, "type": "bf16", "skew": 0.5},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng: random.Random):
    op = rng.choice(("quantise", "product", "grouped"))
    kind = rng.choice(("bf16", "f16", "f32"))
    if op == "quantise":
        while True:
            rows, K = _spread(rng, 1, 32768), _spread(rng, 1, 16384)
            if rows * K <= 8192 * 8192:
                break
        return {"op": op, "rows": rows, "K": K, "type": kind, "stride": rng.choice((0, K + rng.randrange(1, 64)))}
    if op == "product":
        while True:
            M, N, K = _spread(rng, 1, 8192), _spread(rng, 1, 28672), _spread(rng, 32, 16384)
            if M * N * K <= 8192 ** 3 // 2 and N * K <= 28672 * 8192:
                break
        return {"op": op, "M": M, "N": N, "K": K, "type": kind}
    while True:
        T, E, N, K = _spread(rng, 1, 8192), _spread(rng, 1, 128), _spread(rng, 64, 8192), _spread(rng, 64, 8192)
        top = rng.randrange(1, min(E, 8) + 1)
        if E * N * K <= 32 * 4096 * 4096 and T * top * N * K <= 16384 * 4096 * 4096 and E * T * max(N, K) <= 1 << 31:
            break
    return {"op": op, "T": T, "top": top, "E": E, "N": N, "K": K, "type": kind, "skew": rng.choice((0.0, 0.5, 1.0, 2.0))}


# ---- the plain forms -------------------------------------------------------
def _magnitudes(device):
    return torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=device)


def _power(e):
    """2^e in fp32 for whole e in -127 .. 127, from its bits (a power function may be off by one in the last place)."""
    return torch.where(e > -127, (e.int() + 127) << 23, 1 << 22).int().view(torch.float32)


def _plain_quantise(x):
    """(codes, scales) of the rows of x, along the last dimension."""
    K = x.shape[-1]
    x = torch.nn.functional.pad(x.float(), (0, -K % UNIT)).unflatten(-1, (-1, 32))
    largest = x.abs().amax(-1)
    # floor(log2 a) - 2 of the block's largest magnitude: its fraction is in [1/2, 1)
    power = torch.where(largest > 0, torch.frexp(largest)[1] - 3, -127).clamp(-127, 125)
    power = torch.where(torch.arange(power.shape[-1], device=x.device) * 32 >= K, 0, power)  # blocks past the row
    m = (x * _power(-power)[..., None]).abs()
    # nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6; a value between two takes the one of even code
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)
            + 8 * torch.signbit(x)).flatten(-2).to(torch.uint8)
    return code[..., 0::2] | (code[..., 1::2] << 4), (power + 127).to(torch.uint8)


def _plain_values(codes, scales):
    """fp32 values of codes and scales, the padding of the last unit included."""
    nibbles = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()
    v = _magnitudes(codes.device)[nibbles].unflatten(-1, (-1, 32))
    return (v * _power(scales.int() - 127)[..., None]).flatten(-2)


def _plain_product(s):
    return (_plain_values(s["a"], s["sa"]) @ _plain_values(s["b"], s["sb"]).t()).to(s["type"])


def _plain_grouped(s):
    # every expert's rows side by side, as columns padded to the fullest expert's, then one batched product
    x = _plain_values(s["a"], s["sa"])[s["rows"].long()]
    w = _plain_values(s["b"], s["sb"])
    at = torch.arange(x.shape[0], device=x.device)
    expert = torch.searchsorted(s["offsets"][1:].long(), at, right=True)
    slot = at - s["offsets"].long()[expert]
    padded = torch.zeros(w.shape[0], x.shape[1], s["most"], device=x.device)
    padded[expert, :, slot] = x
    return torch.bmm(w, padded)[expert, :, slot].to(s["type"])


# ---- the cases -------------------------------------------------------------
def _activations(g, rows, K):
    """Hidden states: normal values, every row of its own size, a few channels much larger than the rest."""
    x = torch.randn(rows, K, device="cuda", generator=g)
    x *= torch.exp(0.5 * torch.randn(rows, 1, device="cuda", generator=g))
    return x * torch.where(torch.rand(K, device="cuda", generator=g) < 0.005, 12.0, 1.0)


def _weights(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g) * (1.0 / math.sqrt(shape[-1]))


def _routing(case, seed):
    """The tokens of every expert in turn: (rows, sizes), each token on `top` different experts."""
    g = torch.Generator().manual_seed(seed)
    liking = case["skew"] * torch.randn(case["E"], generator=g)
    scores = liking + -torch.log(-torch.log(torch.rand(case["T"], case["E"], generator=g).clamp(1e-6, 1 - 1e-6)))
    chosen = scores.topk(case["top"], dim=1).indices.reshape(-1)
    order = chosen.argsort(stable=True)
    return (order // case["top"]).int(), torch.bincount(chosen, minlength=case["E"])


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = {"op": case["op"], "type": TYPES[case["type"]]}
    if case["op"] == "quantise":
        rows, K = case["rows"], case["K"]
        x = _activations(g, rows, max(K, case["stride"])).to(s["type"])
        s["x"] = x[:, :K]
    elif case["op"] == "product":
        s["a"], s["sa"] = _plain_quantise(_activations(g, case["M"], case["K"]))
        s["b"], s["sb"] = _plain_quantise(_weights(g, case["N"], case["K"]))
    else:
        s["a"], s["sa"] = _plain_quantise(_activations(g, case["T"], case["K"]))
        s["b"], s["sb"] = _plain_quantise(_weights(g, case["E"], case["N"], case["K"]))
        rows, sizes = _routing(case, seed)
        s["rows"] = rows.cuda()
        s["offsets"] = torch.cat((torch.zeros(1, dtype=torch.int64), sizes.cumsum(0))).int().cuda()
        s["most"] = int(sizes.max())
    return s


def run(s):
    if own:
        import precision_integer_gemm_amd as L
        if s["op"] == "quantise":
            codes, scales = L.lpgemm_mxfp4_quantize(s["x"])
            return L.lpgemm_mxfp4_dequantize(codes, scales, s["x"].shape[1], dtype=torch.bfloat16)
        if s["op"] == "product":
            return L.lpgemm_mxfp4(s["a"], s["sa"], s["b"], s["sb"], dtype=s["type"])
        return L.lpgemm_mxfp4_grouped(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], rows=s["rows"], dtype=s["type"])
    if s["op"] == "quantise":
        codes, scales = _plain_quantise(s["x"])
        return _plain_values(codes, scales)[:, : s["x"].shape[1]].to(torch.bfloat16)
    return _plain_product(s) if s["op"] == "product" else _plain_grouped(s)


def work(case):
    w = WIDTH[case["type"]]
    if case["op"] == "quantise":
        # the rows in, their values out as bf16; a maximum, a scaling and a rounding for each value
        n = case["rows"] * case["K"]
        return {"bytes": n * (w + 2), "flops": 3 * n}
    row = -(-case["K"] // UNIT) * (64 + 4)
    if case["op"] == "product":
        M, N = case["M"], case["N"]
        return {"bytes": row * (M + N) + M * N * w, "flops": 2 * M * N * case["K"]}
    # experts that no token takes need not be read: as many are counted as even routing would reach
    R = case["T"] * case["top"]
    reached = min(case["E"], R, case["E"] * (1 - (1 - case["top"] / case["E"]) ** case["T"]))
    return {"bytes": row * (case["T"] + reached * case["N"]) + R * case["N"] * w + 4 * (R + case["E"] + 1),
            "flops": 2 * R * case["N"] * case["K"]}


# ---- the definitions in 64 bits --------------------------------------------
def _exact_power(e):
    """2^e in fp64, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_values(codes, scales):
    """sign * (m / 2 or (1 + m / 2) 2^(e - 1)) * 2^(s - 127): element k of a row in nibble k % 2 of byte k / 2."""
    out = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        c = ((codes >> (4 * half)) & 15).long()
        e, m = (c >> 1) & 3, (c & 1).double()
        v = torch.where(e == 0, m / 2, (1 + m / 2) * _exact_power(e - 1))
        out[..., half::2] = torch.where(c >= 8, -v, v)
    return out * _exact_power(scales.long() - 127).repeat_interleave(32, -1)


def _exact_round_trip(x):
    """The nearest of the fifteen values to x / S in every block of 32, S the largest power of two with max|x| / S >= 4."""
    K = x.shape[1]
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    out = torch.zeros(x.shape[0], K, dtype=torch.float64, device=x.device)
    for k in range(0, K, 32):
        b = x[:, k:k + 32].double()
        a = b.abs().amax(1, keepdim=True)
        S = _exact_power(torch.floor(torch.log2(torch.where(a > 0, a, 1.0))).clamp(min=-125) - 2)
        S = torch.where(a / S >= 8, 2 * S, torch.where((a / S < 4) & (a > 0), S / 2, S))  # log2 rounds
        v = (b / S).abs()
        hi = torch.searchsorted(grid, v.clamp(max=6).contiguous()).clamp(min=1)
        lo = hi - 1
        below, above = v.clamp(max=6) - grid[lo], grid[hi] - v.clamp(max=6)
        pick = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
        out[:, k:k + 32] = torch.where(b < 0, -grid[pick], grid[pick]) * S
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        return _exact_round_trip(s["x"])
    a, b = _exact_values(s["a"], s["sa"]), _exact_values
    if case["op"] == "product":
        return a @ b(s["b"], s["sb"]).t()
    at = s["offsets"].tolist()
    out = torch.empty(s["rows"].numel(), case["N"], dtype=torch.float64, device=a.device)
    for e in range(case["E"]):
        if at[e + 1] > at[e]:
            out[at[e]:at[e + 1]] = a[s["rows"][at[e]:at[e + 1]].long()] @ b(s["b"][e], s["sb"][e]).t()
    return out
