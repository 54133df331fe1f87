"""Cases of the operators for experts in 4 bits and for decoding: microscaled
4-bit quantisation, products of 4-bit rows and matrices grouped by expert, and
a whole expert layer for a few tokens.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits, rounded once at the end), or, where ``own`` is true, through the
library's entry points.  ``exact`` gives the same outputs from the definitions
in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
_MX4 = 17 / 32   # bytes of a 4-bit element with its share of the scale


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One new token's activations on their way into a 4-bit product, and back.
        dict(name="quantize-1-row", op="quantize", rows=1, columns=2048, dtype="bf16"),
        # A prefill batch's activations.
        dict(name="quantize-16384-rows", op="quantize", rows=16384, columns=2048, dtype="bf16"),
        # 64 experts' first matrices, converted from 32-bit master weights when a model is loaded.
        dict(name="quantize-weights", op="quantize", rows=64 * 1024, columns=2048, dtype="f32"),
        # One new token through its experts' first matrix: weights are read, little is computed.
        dict(name="mx4-product-1-token", op="product", tokens=1, experts=64, top_k=4, inner=2048,
             outer=1024, dtype="bf16", gather=True, skew=0.0, padding=0.0),
        # A decoding batch of 32 sequences: most experts are hit by one to four rows each.
        dict(name="mx4-product-32-tokens", op="product", tokens=32, experts=128, top_k=8, inner=2048,
             outer=1024, dtype="bf16", gather=True, skew=0.0, padding=0.0),
        # A prefill batch, rows gathered from the tokens, groups of very different sizes.
        dict(name="mx4-product-16384", op="product", tokens=16384, experts=64, top_k=8, inner=2048,
             outer=1024, dtype="bf16", gather=True, skew=0.5, padding=0.01),
        # Odd everything, half precision.
        dict(name="mx4-product-odd", op="product", tokens=777, experts=7, top_k=3, inner=1003, outer=517,
             dtype="f16", gather=True, skew=1.0, padding=0.05),
        # Decoding one sequence: a gated layer's whole answer for one new token.
        dict(name="layer-1-token", op="layer", tokens=1, experts=64, top_k=4, width=2048, hidden=1024,
             dtype="bf16", mx4=False, gated=True, activation="silu", renormalize=True, padding=0.0),
        # The same with the matrices in 4 bits.
        dict(name="layer-1-token-mx4", op="layer", tokens=1, experts=64, top_k=4, width=2048, hidden=1024,
             dtype="bf16", mx4=True, gated=True, activation="silu", renormalize=True, padding=0.0),
        # Decoding 32 sequences: nearly every expert's matrices are read.
        dict(name="layer-32-tokens", op="layer", tokens=32, experts=128, top_k=8, width=2048, hidden=1024,
             dtype="bf16", mx4=False, gated=True, activation="silu", renormalize=True, padding=0.0),
        # The same with the matrices in 4 bits.
        dict(name="layer-32-tokens-mx4", op="layer", tokens=32, experts=128, top_k=8, width=2048,
             hidden=1024, dtype="bf16", mx4=True, gated=True, activation="silu", renormalize=True,
             padding=0.0),
        # A draft of 13 tokens, odd widths, no gate, half precision, weights over all experts.
        dict(name="layer-odd", op="layer", tokens=13, experts=7, top_k=3, width=1003, hidden=517,
             dtype="f16", mx4=False, gated=False, activation="relu", renormalize=False, padding=0.1),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "layer", "layer"])
    if op == "quantize":
        columns = _log_int(rng, 32, 4096)
        case = dict(op=op, rows=_log_int(rng, 1, 65536), columns=columns,
                    dtype=rng.choice(["bf16", "f16", "f32"]))
        while case["rows"] * columns > 2 ** 27:
            case["rows"] //= 2
        return case
    experts = _log_int(rng, 4, 128)
    top_k = rng.randint(1, min(8, experts))
    if op == "product":
        case = dict(op=op, tokens=_log_int(rng, 1, 16384), experts=experts, top_k=top_k,
                    inner=_log_int(rng, 256, 2048), outer=_log_int(rng, 256, 2048),
                    dtype=rng.choice(["bf16", "f16", "f32"]), gather=rng.random() < 0.5,
                    skew=rng.choice([0.0, 0.5, 1.0]), padding=rng.choice([0.0, 0.05]))
        if rng.random() < 0.75:      # most widths are multiples of 8, the rest are as drawn
            case["inner"] = (case["inner"] + 7) // 8 * 8
            case["outer"] = (case["outer"] + 7) // 8 * 8
        while work(case)["flops"] > 5e11:
            case["tokens"] //= 2
        return case
    case = dict(op=op, tokens=rng.choice([1, _log_int(rng, 1, 64)]), experts=experts, top_k=top_k,
                width=_log_int(rng, 256, 2048), hidden=_log_int(rng, 128, 1024),
                dtype=rng.choice(["bf16", "f16"]), mx4=rng.random() < 0.5, gated=rng.random() < 0.5,
                activation=rng.choice(["silu", "relu"]), renormalize=rng.random() < 0.5,
                padding=rng.choice([0.0, 0.1]))
    if rng.random() < 0.75:
        case["width"] = (case["width"] + 7) // 8 * 8
        case["hidden"] = (case["hidden"] + 7) // 8 * 8
    while work(case)["bytes"] > 1.3e9:
        case["tokens"] //= 2
    return case


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFF)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _matrices(g, experts, outer, inner, dtype, mx4):
    """Each expert's matrix, as 16-bit elements or as 4-bit values and scales."""
    if not mx4:
        w = torch.empty(experts, outer, inner, dtype=dtype, device="cuda")
        for i in range(experts):
            w[i] = _randn(g, outer, inner) / math.sqrt(inner)
        return w
    quads = (inner + 127) // 128
    values = torch.empty(experts, outer, quads * 64, dtype=torch.uint8, device="cuda")
    scales = torch.empty(experts, outer, quads * 4, dtype=torch.uint8, device="cuda")
    for i in range(experts):
        values[i], scales[i] = _quantize(_randn(g, outer, inner) / math.sqrt(inner))
    return values, scales


def _chosen(g, tokens, experts, top_k, skew, padding):
    """Expert ids [tokens, top_k] of distinct experts, -1 for padding tokens."""
    bias = _randn(g, experts) * skew
    noise = -torch.log(-torch.log(torch.rand(tokens, experts, generator=g, device="cuda")
                                  .clamp_(1e-7, 1 - 1e-7)))
    ids = torch.sort(bias + noise, dim=1, descending=True).indices[:, :top_k].to(torch.int32)
    if padding:
        ids[torch.rand(tokens, generator=g, device="cuda") < padding] = -1
    return ids.contiguous()


def _grouped(ids, experts):
    """offsets and order of the flat ids, as routing hands them on."""
    flat = ids.flatten().long()
    key = torch.where(flat < 0, experts, flat)
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    order = torch.where(torch.arange(order.numel(), device="cuda") < offsets[-1], order, -1)
    return offsets.to(torch.int32), order.to(torch.int32)


def prepare(case, seed):
    g = _generator(seed)
    dtype = _DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "quantize":
        # Activations and weights: a few channels are much larger than the rest.
        size = torch.exp(_randn(g, case["columns"]))
        x = torch.empty(case["rows"], case["columns"], dtype=dtype, device="cuda")
        for a in range(0, case["rows"], 16384):
            b = min(a + 16384, case["rows"])
            x[a:b] = _randn(g, b - a, case["columns"]) * size
        s["x"] = x
    elif case["op"] == "product":
        t, k = case["tokens"], case["top_k"]
        ids = _chosen(g, t, case["experts"], k, case["skew"], case["padding"])
        s["offsets"], s["order"] = _grouped(ids, case["experts"])
        s["splits"] = s["offsets"].tolist()
        s["x"] = _randn(g, t if case["gather"] else t * k, case["inner"]).to(dtype)
        s["weight"] = _matrices(g, case["experts"], case["outer"], case["inner"], None, True)
    else:
        t, e, w, h = case["tokens"], case["experts"], case["width"], case["hidden"]
        s["x"] = _randn(g, t, w).to(dtype)
        s["logits"] = _randn(g, t, e)
        if case["padding"]:
            s["logits"][torch.rand(t, generator=g, device="cuda") < case["padding"]] = -math.inf
        s["up"] = _matrices(g, e, h, w, dtype, case["mx4"])
        s["gate"] = _matrices(g, e, h, w, dtype, case["mx4"]) if case["gated"] else None
        s["down"] = _matrices(g, e, w, h, dtype, case["mx4"])
    return s


# ---------------------------------------------------------------- the operators

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import cluster_distributed_shared_gb300 as dh
    case = s["case"]
    if case["op"] == "quantize":
        values, scales = dh.dsmem_mx4_quantize(s["x"])
        return dh.dsmem_mx4_dequantize(values, scales, case["columns"], dtype=s["x"].dtype)
    if case["op"] == "product":
        rows = dict(order=s["order"], fan=case["top_k"]) if case["gather"] else {}
        return dh.dsmem_mx4_grouped_matmul(dh.dsmem_mx4_quantize(s["x"]), s["weight"], s["offsets"],
                                           out_dtype=s["x"].dtype, **rows)
    return dh.dsmem_expert_layer(s["x"], s["logits"], s["up"], s["down"], case["top_k"], gate=s["gate"],
                                 activation=case["activation"], renormalize=case["renormalize"])


def _run_plain(s):
    case = s["case"]
    if case["op"] == "quantize":
        out = torch.empty_like(s["x"])
        for a in range(0, case["rows"], 16384):
            b = a + 16384
            out[a:b] = _dequantize(*_quantize(s["x"][a:b]), case["columns"]).to(out.dtype)
        return out
    if case["op"] == "product":
        return _plain_product(s, case)
    return _plain_layer(s, case)


def _quantize(x):
    """4-bit values, two a byte, and a scale byte of each 32 elements."""
    x = x.float()
    rows, columns = x.shape
    padded = torch.zeros(rows, (columns + 127) // 128 * 128, device=x.device)
    padded[:, :columns] = x
    blocks = padded.view(rows, -1, 32)
    size = blocks.abs()
    most = size.max(dim=2, keepdim=True).values
    exponent = torch.frexp(most).exponent - 1 - 2                 # floor(log2) - 2
    exponent = torch.where(most > 0, exponent, -127).clamp(min=-127)
    # The division by a power of two in two exact steps, either of which 32 bits hold.
    half = torch.div(exponent, 2, rounding_mode="floor")
    v = size * torch.exp2(-half.float()) * torch.exp2((half - exponent).float())
    code = ((v > 0.25).int() + (v >= 0.75).int() + (v > 1.25).int() + (v >= 1.75).int()
            + (v > 2.5).int() + (v >= 3.5).int() + (v > 5.0).int())
    code = code + 8 * torch.signbit(blocks).int()
    code = code.view(rows, -1)
    values = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)
    return values, (exponent + 127).view(rows, -1).to(torch.uint8)


def _dequantize(values, scales, columns):
    """The values that 4-bit tensors stand for, in 32 bits."""
    size = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=values.device)
    table = torch.cat([size, -size])
    low, high = table[(values & 15).int()], table[(values >> 4).int()]
    each = torch.stack([low, high], dim=-1).flatten(-2)
    scale = torch.exp2(scales.float() - 127.0)
    return (each.unflatten(-1, (-1, 32)) * scale.unsqueeze(-1)).flatten(-2)[..., :columns]


def _plain_product(s, case):
    inner, at = case["inner"], s["splits"]
    x = _dequantize(*_quantize(s["x"]), inner)
    values, scales = s["weight"]
    n = s["order"].numel()
    rows = torch.where(s["order"] < 0, 0, s["order"] // case["top_k"]).long() if case["gather"] else None
    y = torch.zeros(n, case["outer"], dtype=s["x"].dtype, device="cuda")
    for i in range(case["experts"]):
        a, b = at[i], at[i + 1]
        if b > a:
            w = _dequantize(values[i], scales[i], inner)
            y[a:b] = ((x[a:b] if rows is None else x[rows[a:b]]) @ w.t()).to(y.dtype)
    return y


def _plain_chosen(s, case):
    """ids and weights of the `top_k` largest logits, as dsmem_route gives them."""
    k, e = case["top_k"], case["experts"]
    logits = s["logits"]
    index = torch.arange(e, device="cuda", dtype=torch.int32)
    left, ids = logits.clone(), []
    for _ in range(k):
        best = left.max(dim=1, keepdim=True).values
        first = torch.where((left == best) & (left > -math.inf), index, e).min(dim=1).values
        ids.append(torch.where(first < e, first, -1))
        left = torch.where(index == first[:, None], -math.inf, left)
    ids = torch.stack(ids, 1)
    found, at = ids >= 0, ids.clamp(min=0).long()
    top = logits.max(dim=1, keepdim=True).values
    top = torch.where(top > -math.inf, top, 0.0)
    raised = torch.exp(logits - top)
    chosen = torch.where(found, raised.gather(1, at), 0.0)
    below = (chosen if case["renormalize"] else raised).sum(dim=1, keepdim=True)
    return at, chosen / torch.where(below > 0, below, 1.0)


def _plain_layer(s, case):
    at, weights = _plain_chosen(s, case)

    def times(matrices, chosen, vectors, columns):
        """Each token's vector times its expert's matrix."""
        if case["mx4"]:
            m = _dequantize(matrices[0][chosen], matrices[1][chosen], columns)
        else:
            m = matrices[chosen].float()
        return torch.bmm(m, vectors.unsqueeze(2)).squeeze(2)

    x = s["x"].float()
    y = torch.zeros_like(x)
    for j in range(case["top_k"]):
        h = times(s["up"], at[:, j], x, case["width"])
        first = times(s["gate"], at[:, j], x, case["width"]) if case["gated"] else h
        active = first / (1.0 + torch.exp(-first)) if case["activation"] == "silu" \
            else torch.where(first > 0, first, 0.0)
        h = active * h if case["gated"] else active
        y = y + weights[:, j:j + 1] * times(s["down"], at[:, j], h, case["hidden"])
    return y.to(s["x"].dtype)


# ---------------------------------------------------------------- work

def _active(case):
    """How many experts a batch's tokens choose, on the average."""
    t = case["tokens"] * (1.0 - case["padding"])
    return case["experts"] * (1.0 - (1.0 - case["top_k"] / case["experts"]) ** t)


def work(case):
    size = _SIZE[case["dtype"]]
    if case["op"] == "quantize":
        n = case["rows"] * case["columns"]
        return dict(bytes=int(2 * n * (size + _MX4)), flops=4 * n)
    pairs = case["tokens"] * case["top_k"]
    if case["op"] == "product":
        rows = pairs * (1.0 - case["padding"])
        source = (case["tokens"] if case["gather"] else pairs) * case["inner"]
        matrix = case["inner"] * case["outer"] * _MX4
        total = source * (size + 2 * _MX4) + _active(case) * matrix + pairs * case["outer"] * size \
            + 4 * (case["experts"] + 1) + (4 * pairs if case["gather"] else 0)
        return dict(bytes=int(total), flops=int(2 * rows * case["inner"] * case["outer"]))
    matrix = case["width"] * case["hidden"] * (3 if case["gated"] else 2)
    total = _active(case) * matrix * (_MX4 if case["mx4"] else 2) \
        + case["tokens"] * (2 * case["width"] * size + 4 * case["experts"])
    return dict(bytes=int(total), flops=int(2 * pairs * (1.0 - case["padding"]) * matrix))


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"quantize": _exact_quantize, "product": _exact_product, "layer": _exact_layer}[case["op"]](s, case)


def _exact_rounded(x):
    """The values to which quantisation takes 64-bit x [rows, columns]."""
    rows, columns = x.shape
    blocks = torch.nn.functional.pad(x, (0, -columns % 32)).view(rows, -1, 32)
    most = blocks.abs().amax(2, keepdim=True)
    scale = torch.ldexp(torch.ones_like(most), torch.frexp(most).exponent - 3)
    scale = torch.where(most > 0, scale, 1.0).clamp(min=2.0 ** -127)
    v = blocks / scale
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
    v = (torch.round(v / step) * step).clamp(-6, 6)        # to even multiples of the step
    return (v * scale).view(rows, -1)[:, :columns]


def _exact_of(matrix, columns):
    """A 4-bit matrix's values in 64 bits, from sign, exponent and fraction of each element."""
    values, scales = (t.to(torch.int64) for t in matrix)
    code = torch.stack([values % 16, values // 16], -1).flatten(-2)
    exponent, fraction = code // 2 % 4, code % 2
    size = torch.where(exponent > 0, (2 + fraction) * 2.0 ** (exponent - 2).double(), fraction * 0.5)
    scale = torch.repeat_interleave(2.0 ** (scales - 127).double(), 32, -1)
    return torch.where(code >= 8, -size, size)[..., :columns] * scale[..., :columns]


def _exact_quantize(s, case):
    return torch.cat([_exact_rounded(part.double()) for part in s["x"].split(8192)])


def _exact_product(s, case):
    at, n, inner = s["splits"], s["order"].numel(), case["inner"]
    x = _exact_rounded(s["x"].double())
    source = s["order"].long() // case["top_k"] if case["gather"] else torch.arange(n, device="cuda")
    y = torch.zeros(n, case["outer"], dtype=torch.float64, device="cuda")
    for i in range(case["experts"]):
        if at[i + 1] > at[i]:
            w = _exact_of((s["weight"][0][i], s["weight"][1][i]), inner)
            y[at[i]:at[i + 1]] = torch.einsum("mk,nk->mn", x.index_select(0, source[at[i]:at[i + 1]]), w)
    return y


def _exact_layer(s, case):
    k = case["top_k"]
    logits = s["logits"].double()
    best = torch.sort(logits, dim=1, descending=True, stable=True)
    p = torch.nan_to_num(torch.softmax(logits, dim=1), nan=0.0).gather(1, best.indices)[:, :k]
    if case["renormalize"]:
        p = torch.nan_to_num(p / p.sum(1, keepdim=True), nan=0.0)
    ids = torch.where(best.values[:, :k] > -math.inf, best.indices[:, :k], -1).tolist()
    x = s["x"].double()
    y = torch.zeros_like(x)

    def matrix(name, e, columns):
        m = s[name]
        return _exact_of((m[0][e], m[1][e]), columns) if case["mx4"] else m[e].double()

    for e in range(case["experts"]):
        where = [(t, j) for t, row in enumerate(ids) for j, i in enumerate(row) if i == e]
        if not where:
            continue
        t, j = torch.tensor(where, device="cuda").t()
        h = x[t] @ matrix("up", e, case["width"]).t()
        first = x[t] @ matrix("gate", e, case["width"]).t() if case["gated"] else h
        active = first * torch.sigmoid(first) if case["activation"] == "silu" else first.clamp(min=0)
        h = active * h if case["gated"] else active
        y[t] += p[t, j, None] * (h @ matrix("down", e, case["hidden"]).t())
    return y
