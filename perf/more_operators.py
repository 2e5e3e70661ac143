"""A layer of routed experts in 8-bit floats as a user's program calls it, with plain forms of each operator.

Five paths: `route` chooses each token's experts from a router's logits and lists
every expert's tokens (a training step: and takes the weights' gradient back to
the logits); `quantise` takes rows to e4m3 codes with one scale per 128 values,
or per 128 x 128, and back; `product` multiplies two such matrices; `grouped`
multiplies the rows routed to each expert by that expert's matrix; `combine`
adds a token's experts up (a training step: and both gradients).  With `own`
false everything is computed with elementary torch operations, in 32 bits, and
in 64 where scores are compared.
"""
import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
WIDTH = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 128  # values of a row that share a scale


def listed():
    return [
        # one token through a router with a bias for balance and four of eight groups: the smallest call, all latency
        {"name": "route-token", "op": "route", "T": 1, "E": 256, "top": 8, "type": "f32", "score": "sigmoid", "bias": True, "groups": 8,
         "top_groups": 4, "group_top": 2, "renormalise": True, "scale": 2.5, "pad": 0, "train": False},
        # a short prompt on many narrow experts, logits as a layer in bf16 leaves them
        {"name": "route-short", "op": "route", "T": 512, "E": 64, "top": 8, "type": "bf16", "score": "softmax", "bias": False, "groups": 1,
         "top_groups": 1, "group_top": 1, "renormalise": True, "scale": 1.0, "pad": 0, "train": False},
        # a training step on a padded batch, with the gradient of the logits
        {"name": "route-train", "op": "route", "T": 8192, "E": 256, "top": 8, "type": "f32", "score": "sigmoid", "bias": True, "groups": 8,
         "top_groups": 4, "group_top": 2, "renormalise": True, "scale": 2.5, "pad": 300, "train": True},
        # a prompt's activations as a slice of a wider buffer: odd length, rows not aligned
        {"name": "quantise-odd-strided", "op": "quantise", "rows": 1001, "K": 2897, "type": "f16", "stride": 2913, "block_rows": 1, "pow2": False},
        # fp32 master weights of a square layer, converted when a model is loaded
        {"name": "quantise-weights-f32", "op": "quantise", "rows": 8192, "K": 8192, "type": "f32", "stride": 0, "block_rows": 128, "pow2": False},
        # decoding a batch of sixteen through an up projection: the weights are read once
        {"name": "product-decode-16", "op": "product", "M": 16, "N": 28672, "K": 8192, "type": "bf16", "block_rows": 128},
        # odd sizes on all sides, both operands with a scale per row and results in fp32, as a weight's gradient is taken
        {"name": "product-odd-f32", "op": "product", "M": 333, "N": 1001, "K": 2897, "type": "f32", "block_rows": 1},
        # the largest: a long prompt through a square layer
        {"name": "product-prompt-8192", "op": "product", "M": 8192, "N": 8192, "K": 8192, "type": "bf16", "block_rows": 128},
        # decoding sixteen tokens, four of thirty-two experts each: most experts have a row or two, some none
        {"name": "grouped-decode", "op": "grouped", "T": 16, "top": 4, "E": 32, "N": 4096, "K": 4096, "type": "bf16", "skew": 1.0, "block_rows": 128},
        # a long prompt, two of thirty-two experts for each token
        {"name": "grouped-prompt", "op": "grouped", "T": 8192, "top": 2, "E": 32, "N": 4096, "K": 4096, "type": "bf16", "skew": 0.5, "block_rows": 128},
        # the same sixteen tokens' experts, added to what the shared expert gave
        {"name": "combine-decode", "op": "combine", "T": 16, "top": 4, "N": 4096, "type": "bf16", "residual": True, "pad": 0, "train": False},
        # a training step on a padded batch of long rows
        {"name": "combine-train", "op": "combine", "T": 8192, "top": 4, "N": 4096, "type": "bf16", "residual": False, "pad": 300, "train": True},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng: random.Random):
    op = rng.choice(("route", "quantise", "product", "grouped", "combine"))
    kind = rng.choice(("bf16", "f16", "f32"))
    if op == "route":
        while True:
            T, groups, size = _spread(rng, 1, 16384), rng.choice((1, 1, 1, 2, 4, 8, 13, 16)), _spread(rng, 1, 512)
            E = groups * size
            if 2 <= E <= 512 and T * E <= 8192 * 512:
                break
        top_groups = rng.randrange(1, groups + 1)
        top = rng.randrange(1, min(16, top_groups * size) + 1)
        return {"op": op, "T": T, "E": E, "top": top, "type": kind, "score": rng.choice(("softmax", "sigmoid")),
                "bias": rng.random() < 0.5, "groups": groups, "top_groups": top_groups, "group_top": rng.choice((1, 2)),
                "renormalise": top > 1 and rng.random() < 0.7,  # one expert's renormalised weight is 1 and has no gradient
                "scale": rng.choice((1.0, 2.5)), "pad": rng.choice((0, T // 10)), "train": rng.random() < 0.5}
    if op == "quantise":
        while True:
            rows, K = _spread(rng, 1, 32768), _spread(rng, 1, 16384)
            if rows * K <= 8192 * 8192:
                break
        return {"op": op, "rows": rows, "K": K, "type": kind, "stride": rng.choice((0, K + rng.randrange(1, 64))), "block_rows": rng.choice((1, 128)),
                "pow2": rng.random() < 0.5}
    if op == "product":
        while True:
            M, N, K = _spread(rng, 1, 8192), _spread(rng, 1, 28672), _spread(rng, 32, 16384)
            if M * N * K <= 8192 ** 3 // 2 and N * K <= 28672 * 8192:
                break
        return {"op": op, "M": M, "N": N, "K": K, "type": kind, "block_rows": rng.choice((1, 128, 128))}
    if op == "grouped":
        while True:
            T, E, N, K = _spread(rng, 1, 8192), _spread(rng, 1, 128), _spread(rng, 64, 8192), _spread(rng, 64, 8192)
            top = rng.randrange(1, min(E, 8) + 1)
            if E * N * K <= 32 * 4096 * 4096 and T * top * N * K <= 16384 * 4096 * 4096 and E * T * max(N, K) <= 1 << 31:
                break
        return {"op": op, "T": T, "top": top, "E": E, "N": N, "K": K, "type": kind, "skew": rng.choice((0.0, 0.5, 1.0, 2.0)), "block_rows": rng.choice((1, 128, 128))}
    while True:
        T, top, N = _spread(rng, 1, 16384), rng.randrange(1, 9), _spread(rng, 1, 8192)
        if T * top * N <= 8192 * 4 * 4096:
            break
    return {"op": op, "T": T, "top": top, "N": N, "type": kind, "residual": rng.random() < 0.5, "pad": rng.choice((0, T // 10)), "train": rng.random() < 0.5}


# ---- the plain forms -------------------------------------------------------
def _blocks(x):
    """x [.., rows, K] padded to whole blocks along K, as [.., rows, U, 128]."""
    return torch.nn.functional.pad(x, (0, -x.shape[-1] % BLOCK)).unflatten(-1, (-1, BLOCK))


def _by_row(scales, rows, dim):
    """The scale of each row, whether given for it or for its 128 rows."""
    return scales if scales.shape[dim] == rows else scales.repeat_interleave(BLOCK, dim).narrow(dim, 0, rows)


def _plain_quantise(x, block_rows=1, pow2=False):
    """(codes [.., rows, 128 U], scales [.., rows or rows / 128, U]) of the rows of x."""
    rows, x = x.shape[-2], _blocks(x.float())
    a = x.abs().amax(-1)
    if block_rows > 1:
        a = torch.nn.functional.pad(a, (0, 0, 0, -rows % block_rows)).unflatten(-2, (-1, block_rows)).amax(-2)
    low = a.clamp(min=2.0 ** -100)
    if pow2:  # the smallest power of two that leaves at most 448, from the exponent's bits
        fraction, exponent = torch.frexp(low)
        scale = ((exponent - 9 + (fraction > 0.875) + 127) << 23).int().view(torch.float32)
    else:
        scale = low / torch.full_like(low, 448)  # a number in its place would be multiplied by its inverse
    fine = torch.isfinite(a)
    scale = torch.where(fine, scale, float("nan"))
    inverse = torch.where(fine, 1 / scale, 0.0)
    y = torch.where(_by_row(fine, rows, -2)[..., None], x * _by_row(inverse, rows, -2)[..., None], 0.0)
    return y.to(torch.float8_e4m3fn).flatten(-2), scale


def _plain_values(codes, scales):
    """fp32 values of codes and scales, the padding of the last block included."""
    s = _by_row(scales, codes.shape[-2], -2)
    return (codes.float().unflatten(-1, (-1, BLOCK)) * s[..., None]).flatten(-2)


def _scores(s, logits):
    """(score, choice score) of every expert, in 64 bits; a choice score of -inf is closed."""
    x = logits.double()
    closed = x == -math.inf
    if s["score"] == "softmax":
        top = x.amax(1, keepdim=True)
        e = torch.where(closed, 0.0, torch.exp(x - torch.where(top == -math.inf, 0.0, top)))
        p = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        p = torch.where(closed, 0.0, 1 / (1 + torch.exp(-x)))
    if s["bias"] is None and s["group_top"] == 1:
        return p, x  # both scores grow with the logits: no rounding makes a tie
    c = p if s["bias"] is None else p + s["bias"].double()
    return p, torch.where(closed, -math.inf, c)


def _plain_route(s):
    logits, T, E, top = s["logits"], s["logits"].shape[0], s["logits"].shape[1], s["top"]
    p, c = _scores(s, logits)
    if s["top_groups"] < s["groups"]:
        of_group = c.view(T, s["groups"], -1)
        best = of_group.sort(dim=2, descending=True, stable=True).values[:, :, :s["group_top"]]
        score = torch.where(best[:, :, 0] == -math.inf, -math.inf, torch.where(best == -math.inf, 0.0, best).sum(2))
        kept = score.sort(dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        keep = torch.zeros(T, s["groups"], dtype=torch.bool, device=c.device)
        keep[torch.arange(T, device=c.device)[:, None], kept] = True
        c = torch.where(keep[:, :, None], of_group, -math.inf).flatten(1)
    best, experts = c.sort(dim=1, descending=True, stable=True)
    experts = torch.where(best[:, :top] == -math.inf, -1, experts[:, :top])
    there = experts >= 0
    chosen = torch.where(there, p[torch.arange(T, device=c.device)[:, None], experts.clamp(min=0)], 0.0)
    total = chosen.sum(1, keepdim=True)
    weights = chosen / torch.where(total == 0, 1.0, total) if s["renormalise"] else chosen
    weights = (weights * s["scale"]).float()
    flat = torch.where(there, experts, E).flatten()
    order = flat.argsort(stable=True)
    offsets = torch.nn.functional.pad((flat[:, None] == torch.arange(E, device=c.device)).sum(0).cumsum(0), (1, 0))
    rows = torch.where(torch.arange(T * top, device=c.device) < offsets[-1], order // top, -1)
    places = torch.empty_like(flat)
    places[order] = torch.arange(T * top, device=c.device)
    places = torch.where(there, places.view(T, top), -1)
    out = {"experts": experts.int(), "weights": weights, "rows": rows.int(), "offsets": offsets.int(), "places": places.int()}
    if s["train"]:
        out["dlogits"] = _plain_route_gradient(s, p, experts, there, chosen, total).to(logits.dtype)
    return out


def _plain_route_gradient(s, p, experts, there, chosen, total):
    g = torch.where(there, s["dweights"].double() * s["scale"], 0.0)
    if s["renormalise"]:
        total = torch.where(total == 0, math.inf, total)
        g = (g - (g * chosen).sum(1, keepdim=True) / total) / total
    dp = torch.zeros_like(p).scatter_add_(1, experts.clamp(min=0), torch.where(there, g, 0.0))
    if s["score"] == "softmax":
        return p * (dp - (p * dp).sum(1, keepdim=True))
    return p * (1 - p) * dp


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


def _plain_combine(s):
    there = s["places"] >= 0
    picked = s["y"][s["places"].clamp(min=0).long()].float()  # [T, top, N]
    w = torch.where(there, s["weights"], 0.0)
    out = torch.where(there[..., None], w[..., None] * picked, 0.0).sum(1)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    out = out.to(s["type"])
    if not s["train"]:
        return out
    d = s["dout"].float()[:, None]
    dw = torch.where(there, (d * picked).sum(2), 0.0)
    dy = torch.zeros_like(s["y"])
    dy[s["places"][there].long()] = (w[..., None] * d)[there].to(dy.dtype)
    return {"out": out, "dy": dy, "dweights": dw}


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
    s = {k: case[k] for k in case if k not in ("name", "type", "bias", "residual")}
    s["type"] = TYPES[case["type"]]
    if case["op"] == "route":
        T, E = case["T"], case["E"]
        liked = torch.randn(E, device="cuda", generator=g)
        s["logits"] = (1.5 * torch.randn(T, E, device="cuda", generator=g) + 0.5 * liked).to(s["type"])
        s["logits"][T - case["pad"]:] = -math.inf  # the batch's padding goes to no expert
        s["bias"] = -0.1 * liked + 0.02 * torch.randn(E, device="cuda", generator=g) if case["bias"] else None
        s["dweights"] = torch.randn(T, case["top"], device="cuda", generator=g)
    elif case["op"] == "quantise":
        x = _activations(g, case["rows"], max(case["K"], case["stride"])).to(s["type"])
        s["x"] = x[:, :case["K"]]
    elif case["op"] == "product":
        s["a"], s["sa"] = _plain_quantise(_activations(g, case["M"], case["K"]))
        s["b"], s["sb"] = _plain_quantise(_weights(g, case["N"], case["K"]), case["block_rows"])
    elif case["op"] == "grouped":
        s["a"], s["sa"] = _plain_quantise(_activations(g, case["T"], case["K"]))
        s["b"], s["sb"] = _plain_quantise(_weights(g, case["E"], case["N"], case["K"]), case["block_rows"])
        rows, sizes = _routing(case, seed)
        s["rows"] = rows.cuda()
        s["offsets"] = torch.cat((torch.zeros(1, dtype=torch.int64), sizes.cumsum(0))).int().cuda()
        s["most"] = int(sizes.max())
    else:
        T, top, N = case["T"], case["top"], case["N"]
        s["y"] = torch.randn(T * top, N, device="cuda", generator=g).to(s["type"])
        # tokens come back from anywhere among the experts' rows; the padding's are in nobody's
        s["places"] = torch.randperm(T * top, device="cuda", generator=g).int().view(T, top)
        s["places"][T - case["pad"]:] = -1
        w = torch.rand(T, top, device="cuda", generator=g) + 0.1
        s["weights"] = w / w.sum(1, keepdim=True)
        s["residual"] = torch.randn(T, N, device="cuda", generator=g).to(s["type"]) if case["residual"] else None
        if case["train"]:
            s["dout"] = torch.randn(T, N, device="cuda", generator=g).to(s["type"])
            s["dy"] = torch.zeros_like(s["y"])  # rows that are in no token's places stay zero
    return s


def _own(s):
    import precision_integer_gemm_amd as L
    if s["op"] == "route":
        r = L.lpgemm_route(s["logits"], s["top"], score=s["score"], bias=s["bias"], groups=s["groups"], top_groups=s["top_groups"],
                           group_top=s["group_top"], renormalise=s["renormalise"], scale=s["scale"])
        out = {"experts": r.experts, "weights": r.weights, "rows": r.rows, "offsets": r.offsets, "places": r.places}
        if s["train"]:
            out["dlogits"] = L.lpgemm_route_backward(s["dweights"], s["logits"], r.experts, score=s["score"], renormalise=s["renormalise"], scale=s["scale"])
        return out
    if s["op"] == "quantise":
        codes, scales = L.lpgemm_fp8_block_quantize(s["x"], block_rows=s["block_rows"], power_of_two=s["pow2"])
        return L.lpgemm_fp8_block_dequantize(codes, scales, s["x"].shape[1], dtype=torch.bfloat16), scales
    if s["op"] == "product":
        return L.lpgemm_fp8_block(s["a"], s["sa"], s["b"], s["sb"], dtype=s["type"])
    if s["op"] == "grouped":
        return L.lpgemm_fp8_block_grouped(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], rows=s["rows"], dtype=s["type"])
    out = L.lpgemm_combine(s["y"], s["places"], s["weights"], residual=s["residual"])
    if not s["train"]:
        return out
    dy, dw = L.lpgemm_combine_backward(s["dout"], s["y"], s["places"], s["weights"], dy=s["dy"])
    return {"out": out, "dy": dy, "dweights": dw}


def run(s):
    if own:
        return _own(s)
    if s["op"] == "route":
        return _plain_route(s)
    if s["op"] == "quantise":
        codes, scales = _plain_quantise(s["x"], s["block_rows"], s["pow2"])
        return _plain_values(codes, scales)[:, :s["x"].shape[1]].to(torch.bfloat16), scales
    if s["op"] == "product":
        return (_plain_values(s["a"], s["sa"]) @ _plain_values(s["b"], s["sb"]).t()).to(s["type"])
    return _plain_grouped(s) if s["op"] == "grouped" else _plain_combine(s)


def work(case):
    w = WIDTH[case["type"]]
    if case["op"] == "route":
        # logits in, the five lists out; a score and a few comparisons for each expert; training: logits again, their gradient out
        T, E, top = case["T"], case["E"], case["top"]
        n = {"bytes": T * E * w + T * top * 16 + 4 * (E + 1) + (4 * E if case["bias"] else 0), "flops": 6 * T * E}
        if case["train"]:
            n = {"bytes": n["bytes"] + 2 * T * E * w + 4 * T * top, "flops": 2 * n["flops"]}
        return n
    if case["op"] == "quantise":
        # the rows in, their values out as bf16, the scales out; a maximum, a scaling and a rounding for each value
        n, U = case["rows"] * case["K"], -(-case["K"] // BLOCK)
        return {"bytes": n * (w + 2) + 4 * U * -(-case["rows"] // case["block_rows"]), "flops": 3 * n}
    if case["op"] == "combine":
        T, top, N = case["T"], case["top"], case["N"]
        R, t = (T - case["pad"]) * top, case["train"]
        n = R * N * w + T * N * w * (2 if case["residual"] else 1) + 8 * T * top
        # training: the rows and the gradient again, the rows' gradient out
        return {"bytes": n + (2 * R * N * w + T * N * w + 12 * T * top if t else 0), "flops": (5 if t else 2) * R * N}
    U = -(-case["K"] // BLOCK)
    row, scales = U * BLOCK, lambda n: 4 * U * -(-n // case["block_rows"])
    if case["op"] == "product":
        M, N = case["M"], case["N"]
        return {"bytes": row * (M + N) + 4 * U * M + scales(N) + M * N * w, "flops": 2 * M * N * case["K"]}
    # experts that no token takes need not be read: as many are counted as even routing would reach
    R = case["T"] * case["top"]
    reached = min(case["E"], R, case["E"] * (1 - (1 - case["top"] / case["E"]) ** case["T"]))
    return {"bytes": (row + 4 * U) * case["T"] + reached * (row * case["N"] + scales(case["N"])) + R * case["N"] * w + 4 * (R + case["E"] + 1),
            "flops": 2 * R * case["N"] * case["K"]}


# ---- the definitions in 64 bits --------------------------------------------
def _exact_code_values(codes):
    """(-1)^s (m / 8) 2^-6 or (-1)^s (1 + m / 8) 2^(e - 7) of e4m3 bytes s eeee mmm."""
    c = codes.view(torch.uint8).long()
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m / 512, (8 + m) * ((e + 1023 - 10) << 52).view(torch.float64))
    return torch.where(c >= 128, -v, v)


def _exact_values(codes, scales):
    v = _exact_code_values(codes).unflatten(-1, (-1, BLOCK))
    s = scales.double()
    if s.shape[-2] != v.shape[-3]:
        s = s[..., torch.arange(v.shape[-3], device=s.device) // BLOCK, :]
    return (v * s[..., None]).flatten(-2)


def _exact_round_trip(case, x):
    """Blocks of 128 columns, of one row or 128: the nearest of e4m3's values to each value over the block's scale."""
    grid = _exact_code_values(torch.arange(127, dtype=torch.uint8, device=x.device))
    rows, K = x.shape
    R = case["block_rows"]
    out = torch.empty(rows, K, dtype=torch.float64, device=x.device)
    scales = torch.empty(-(-rows // R), -(-K // BLOCK), dtype=torch.float64, device=x.device)
    group = torch.arange(rows, device=x.device) // R
    for j in range(scales.shape[1]):
        b = x[:, BLOCK * j:BLOCK * (j + 1)].double()
        a = torch.zeros(scales.shape[0], dtype=torch.float64, device=x.device).scatter_reduce(0, group, b.abs().amax(1), "amax").clamp(min=2.0 ** -100)
        if case["pow2"]:
            up = torch.ceil(torch.log2(a / 448))
            up = torch.where(a / 448 > torch.exp2(up), up + 1, torch.where(a / 448 <= torch.exp2(up - 1), up - 1, up))  # log2 rounds
            s = torch.exp2(up.round())
        else:
            s = (a / 448).float().double()  # the scale is a number of 32 bits
        scales[:, j] = s
        inverse = (1 / s).float().double()[group][:, None]  # and so are its inverse and the scaled value
        v = (b * inverse).float().double()
        near = torch.searchsorted(grid, v.abs().clamp(max=448).contiguous()).clamp(min=1, max=126)
        below, above = v.abs().clamp(max=448) - grid[near - 1], grid[near] - v.abs().clamp(max=448)
        pick = torch.where((below < above) | ((below == above) & (near % 2 == 1)), near - 1, near)
        out[:, BLOCK * j:BLOCK * (j + 1)] = torch.where(b < 0, -grid[pick], grid[pick]) * s[group][:, None]
    return out, scales


def _exact_route(case, s):
    """Scores, weights and gradient in 64 bits, the experts one after another: the best that is left, the first of equal ones."""
    x = s["logits"].double()
    T, E = x.shape
    open_ = x > -math.inf
    if case["score"] == "softmax":
        p = torch.softmax(torch.where(open_.any(1, keepdim=True), x, 0.0), 1)
    else:
        p = torch.sigmoid(x)
    p = torch.where(open_, p, 0.0)
    by_logits = not case["bias"] and case["group_top"] == 1
    c = x.clone() if by_logits else torch.where(open_, p + (s["bias"].double() if case["bias"] else 0.0), -math.inf)

    def take(values, n):  # the places of the n largest of each row, in order
        left, got = values.clone(), []
        at = torch.arange(left.shape[1], device=x.device)
        for _ in range(n):
            most = left.amax(1, keepdim=True)
            first = torch.where(left == most, at, left.shape[1]).amin(1)
            got.append(torch.where(most[:, 0] > -math.inf, first, -1))
            left[torch.arange(T, device=x.device), first] = -math.inf
        return torch.stack(got, 1)

    if case["top_groups"] < case["groups"]:
        size = E // case["groups"]
        score = torch.empty(T, case["groups"], dtype=torch.float64, device=x.device)
        for i in range(case["groups"]):
            part = c[:, i * size:(i + 1) * size]
            at = take(part, min(case["group_top"], size))
            v = part.gather(1, at.clamp(min=0))
            score[:, i] = torch.where(at[:, 0] < 0, -math.inf, torch.where(at >= 0, v, 0.0).sum(1))
        kept = take(score, case["top_groups"])
        allowed = (kept[:, :, None] == (torch.arange(E, device=x.device) // size)).any(1)
        c = torch.where(allowed, c, -math.inf)
    experts = take(c, case["top"])
    there = experts >= 0
    chosen = torch.where(there, p.gather(1, experts.clamp(min=0)), 0.0)
    total = chosen.sum(1, keepdim=True) if case["renormalise"] else torch.ones(T, 1, dtype=torch.float64, device=x.device)
    share = torch.where(total > 0, chosen / total, 0.0)
    sizes = torch.bincount(experts[there], minlength=E)
    offsets = torch.cat((sizes.new_zeros(1), sizes.cumsum(0)))
    rows = torch.full((T * case["top"],), -1, dtype=torch.int64, device=x.device)
    places = torch.full((T, case["top"]), -1, dtype=torch.int64, device=x.device)
    token, slot = there.nonzero(as_tuple=True)
    order = (experts[there] * T + token).argsort()
    rows[:order.numel()] = token[order]
    places[token[order], slot[order]] = torch.arange(order.numel(), device=x.device)
    out = {"experts": experts.int(), "weights": case["scale"] * share, "rows": rows.int(), "offsets": offsets.int(), "places": places.int()}
    if case["train"]:
        dw = s["dweights"].double()
        # d weight_k / d p_i = scale (delta_ki - share_k) / total, without the second term where nothing is renormalised
        back = dw - (dw * share).sum(1, keepdim=True) if case["renormalise"] else dw
        dp = torch.zeros_like(p)
        token, slot = there.nonzero(as_tuple=True)
        dp[token, experts[there]] = torch.where(total > 0, case["scale"] * back / total, 0.0)[there]
        mean = (dp * p).sum(1, keepdim=True)
        out["dlogits"] = dp * p - p * mean if case["score"] == "softmax" else dp * p * (1 - p)
    return out


def _exact_combine(case, s):
    T = case["T"]
    out = s["residual"].double() if s["residual"] is not None else torch.zeros(T, case["N"], dtype=torch.float64, device=s["y"].device)
    dy, dw = torch.zeros(s["y"].shape, dtype=torch.float64, device=out.device), torch.zeros(T, case["top"], dtype=torch.float64, device=out.device)
    for k in range(case["top"]):
        t = (s["places"][:, k] >= 0).nonzero()[:, 0]
        i, w = s["places"][t, k].long(), s["weights"][t, k].double()[:, None]
        y = s["y"][i].double()
        out[t] += w * y
        if case["train"]:
            d = s["dout"][t].double()
            dw[t, k] = (d * y).sum(1)
            dy[i] = w * d
    return {"out": out, "dy": dy, "dweights": dw} if case["train"] else out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "quantise":
        return _exact_round_trip(case, s["x"])
    if case["op"] == "combine":
        return _exact_combine(case, s)
    a = _exact_values(s["a"], s["sa"])
    if case["op"] == "product":
        return a @ _exact_values(s["b"], s["sb"]).t()
    at = s["offsets"].tolist()
    out = torch.empty(s["rows"].numel(), case["N"], dtype=torch.float64, device=a.device)
    for e in range(case["E"]):
        if at[e + 1] > at[e]:
            out[at[e]:at[e + 1]] = a[s["rows"][at[e]:at[e + 1]].long()] @ _exact_values(s["b"][e], s["sb"][e]).t()
    return out
