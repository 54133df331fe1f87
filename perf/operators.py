"""Cases of the expert-layer operators: routing, products grouped by expert,
the weighted way back, and the gradients' global norm with clipping.

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


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One new token of one sequence: the router's latency while serving.
        dict(name="route-1-of-64", op="route", tokens=1, experts=64, top_k=4, dtype="f32",
             renormalize=True, backward=False, padding=0.0, masked=0),
        # A training batch of 16384 tokens (2% padding, every expert masked there), gradient included.
        dict(name="route-16384-of-256-train", op="route", tokens=16384, experts=256, top_k=8,
             dtype="f32", renormalize=True, backward=True, padding=0.02, masked=0),
        # One new token through its experts' first matrix: weights are read, little is computed.
        dict(name="product-1-token", op="product", kind="forward", tokens=1, experts=64, top_k=4,
             inner=2048, outer=1024, dtype="bf16", gather=True, skew=0.0, padding=0.0),
        # A decoding batch of 32 sequences: most experts are hit by one to four rows each.
        dict(name="product-32-tokens", op="product", kind="forward", tokens=32, experts=128, top_k=8,
             inner=2048, outer=1024, dtype="bf16", gather=True, skew=0.0, padding=0.0),
        # A training batch, rows gathered from the tokens, groups of very different sizes.
        dict(name="product-16384-forward", op="product", kind="forward", tokens=16384, experts=64,
             top_k=8, inner=2048, outer=1024, dtype="bf16", gather=True, skew=0.5, padding=0.01),
        # The same batch's gradient with respect to the rows.
        dict(name="product-16384-input-gradient", op="product", kind="input_gradient", tokens=16384,
             experts=64, top_k=8, inner=2048, outer=1024, dtype="bf16", gather=False, skew=0.5,
             padding=0.01),
        # The same batch's gradient with respect to the experts' matrices: ragged sums.
        dict(name="product-16384-weight-gradient", op="product", kind="weight_gradient", tokens=16384,
             experts=64, top_k=8, inner=2048, outer=1024, dtype="bf16", gather=True, skew=0.5,
             padding=0.01),
        # Odd everything, half precision, all three products of a small training step.
        dict(name="product-odd-step", op="product", kind="step", tokens=777, experts=7, top_k=3,
             inner=1003, outer=517, dtype="f16", gather=True, skew=1.0, padding=0.05),
        # The experts' answers of a decoding batch, weighted and summed.
        dict(name="combine-16-tokens", op="combine", tokens=16, experts=64, top_k=4, width=2048,
             dtype="bf16", backward=False, padding=0.0),
        # The same for a training batch, with the gradients of rows and weights.
        dict(name="combine-16384-train", op="combine", tokens=16384, experts=64, top_k=8, width=2048,
             dtype="bf16", backward=True, padding=0.01),
        # Gradients of a small model: few tensors, odd sizes, both precisions.
        dict(name="clip-small", op="clip", tensors=37, elements=3_000_001, dtype="mixed",
             magnitude=1.0),
        # Gradients of a layer stack with experts: hundreds of tensors, half a billion values.
        dict(name="clip-large", op="clip", tensors=291, elements=500_000_000, dtype="bf16",
             magnitude=1.0),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["route", "product", "product", "combine", "clip"])
    if op == "route":
        experts = _log_int(rng, 4, 256)
        return dict(op=op, tokens=_log_int(rng, 1, 16384), experts=experts,
                    top_k=rng.randint(1, min(8, experts)), dtype=rng.choice(["f32", "bf16", "f16"]),
                    renormalize=rng.random() < 0.5, backward=rng.random() < 0.5,
                    padding=rng.choice([0.0, 0.05]), masked=rng.choice([0, 0, 1, experts // 3]))
    if op == "product":
        experts = _log_int(rng, 4, 128)
        case = dict(op=op,
                    kind=rng.choice(["forward", "forward", "input_gradient", "weight_gradient", "step"]),
                    tokens=_log_int(rng, 1, 8192), experts=experts,
                    top_k=rng.randint(1, min(8, experts)), inner=_log_int(rng, 256, 2048),
                    outer=_log_int(rng, 256, 2048), dtype=rng.choice(["bf16", "f16"]),
                    gather=rng.random() < 0.5, skew=rng.choice([0.0, 0.5, 1.0]),
                    padding=rng.choice([0.0, 0.05]))
        if rng.random() < 0.75:      # most widths are multiples of 8, the rest are as drawn
            case["inner"] = (case["inner"] + 7) // 8 * 8
            case["outer"] = (case["outer"] + 7) // 8 * 8
        while work(case)["flops"] > 5e11:
            case["tokens"] //= 2
        return case
    if op == "combine":
        experts = _log_int(rng, 4, 128)
        return dict(op=op, tokens=_log_int(rng, 1, 16384), experts=experts,
                    top_k=rng.randint(1, min(8, experts)), width=_log_int(rng, 256, 2048),
                    dtype=rng.choice(["bf16", "f16", "f32"]), backward=rng.random() < 0.5,
                    padding=rng.choice([0.0, 0.05]))
    tensors = _log_int(rng, 1, 400)
    return dict(op=op, tensors=tensors, elements=_log_int(rng, 1000 * tensors, 200_000_000),
                dtype=rng.choice(["bf16", "f16", "f32", "mixed"]), magnitude=rng.choice([1e-3, 1.0]))


# ---------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFF)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


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
    """offsets, order, position of the flat ids, as routing hands them on."""
    flat = ids.flatten().long()
    key = torch.where(flat < 0, experts, flat)
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device="cuda")
    position = torch.where(flat < 0, -1, position)
    order = torch.where(torch.arange(order.numel(), device="cuda") < offsets[-1], order, -1)
    return offsets.to(torch.int32), order.to(torch.int32), position.to(torch.int32)


def _clip_shapes(case):
    """Element counts of the tensors: a few large, most of middle size, some tiny and odd."""
    n, total = case["tensors"], case["elements"]
    share = [((i * 2654435761) % 1009 + 1) ** 3 for i in range(n)]
    scale = total / sum(share)
    return [max(1, int(s * scale)) for s in share]


def _clip_dtypes(case):
    if case["dtype"] != "mixed":
        return [case["dtype"]] * case["tensors"]
    return [("bf16", "f32")[i % 2] for i in range(case["tensors"])]


def _buckets(tensors):
    """One flat bucket for each dtype, and in it a view for each tensor: the clipped gradients as a
    reduction over ranks takes them.  Views begin at multiples of 64 elements."""
    ends, starts = {}, []
    for t in tensors:
        starts.append(ends.get(t.dtype, 0))
        ends[t.dtype] = starts[-1] + (t.numel() + 63) // 64 * 64
    flat = {d: torch.zeros(n, dtype=d, device=tensors[0].device) for d, n in ends.items()}
    return list(flat.values()), [flat[t.dtype][a:a + t.numel()] for a, t in zip(starts, tensors)]


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=case)
    if case["op"] == "route":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        logits = _randn(g, t, e) + 0.5 * _randn(g, e)
        if case["masked"]:
            logits[:, torch.randperm(e, generator=g, device="cuda")[:case["masked"]]] = -math.inf
        if case["padding"]:
            logits[torch.rand(t, generator=g, device="cuda") < case["padding"]] = -math.inf
        s["logits"] = logits.to(_DTYPES[case["dtype"]])
        s["grad_weights"] = _randn(g, t, k)
    elif case["op"] == "product":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        inner, outer, dtype = case["inner"], case["outer"], _DTYPES[case["dtype"]]
        ids = _chosen(g, t, e, k, case["skew"], case["padding"])
        s["offsets"], s["order"], _ = _grouped(ids, e)
        s["splits"] = s["offsets"].tolist()
        n = t * k
        if case["kind"] != "weight_gradient":
            s["weight"] = torch.empty(e, outer, inner, dtype=dtype, device="cuda")
            for i in range(e):
                s["weight"][i] = _randn(g, outer, inner) / math.sqrt(inner)
        if case["kind"] != "input_gradient":
            s["x"] = _randn(g, t if case["gather"] else n, inner).to(dtype)
        if case["kind"] != "forward":
            s["dy"] = _randn(g, n, outer).to(dtype)
    elif case["op"] == "combine":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        ids = _chosen(g, t, e, k, 0.0, case["padding"])
        _, s["order"], position = _grouped(ids, e)
        s["position"] = position.view(t, k)
        s["weights"] = torch.softmax(_randn(g, t, k), 1) * (ids >= 0)
        s["z"] = _randn(g, t * k, case["width"]).to(_DTYPES[case["dtype"]])
        if case["backward"]:
            s["dy"] = _randn(g, t, case["width"]).to(_DTYPES[case["dtype"]])
    else:
        s["grads"] = [(_randn(g, size) * case["magnitude"]).to(_DTYPES[d])
                      for size, d in zip(_clip_shapes(case), _clip_dtypes(case))]
        s["buckets"], s["clipped"] = _buckets(s["grads"])
        s["max_norm"] = 1.0
    return s


# ---------------------------------------------------------------- the operators

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import cluster_distributed_shared_gb300 as dh
    case = s["case"]
    if case["op"] == "route":
        ids, weights = dh.dsmem_route(s["logits"], case["top_k"], renormalize=case["renormalize"])
        offsets, order, position = dh.dsmem_group(ids, case["experts"])
        out = [ids, weights, offsets, order, position]
        if case["backward"]:
            out.append(dh.dsmem_route_backward(s["logits"], ids, weights, s["grad_weights"],
                                               renormalize=case["renormalize"]))
        return out
    if case["op"] == "product":
        rows = dict(order=s["order"], fan=case["top_k"]) if case["gather"] else {}
        out = []
        if case["kind"] in ("forward", "step"):
            out.append(dh.dsmem_grouped_matmul(s["x"], s["weight"], s["offsets"], **rows))
        if case["kind"] in ("input_gradient", "step"):
            out.append(dh.dsmem_grouped_matmul(s["dy"], s["weight"], s["offsets"], transpose=True))
        if case["kind"] in ("weight_gradient", "step"):
            out.append(dh.dsmem_grouped_matmul_wgrad(s["dy"], s["x"], s["offsets"], **rows))
        return out
    if case["op"] == "combine":
        out = [dh.dsmem_combine(s["z"], s["position"], s["weights"])]
        if case["backward"]:
            out += dh.dsmem_combine_backward(s["dy"], s["z"], s["position"], s["order"],
                                             s["weights"])
        return out
    norm = dh.dsmem_grad_clip(s["grads"], s["max_norm"], out=s["clipped"])
    return [norm, *s["buckets"]]


def _run_plain(s):
    case = s["case"]
    if case["op"] == "route":
        return _plain_route(s, case)
    if case["op"] == "product":
        return _plain_product(s, case)
    if case["op"] == "combine":
        return _plain_combine(s, case)
    total = torch.zeros((), device="cuda")
    for t in s["grads"]:
        v = t.float()
        total = total + (v * v).sum()
    norm = torch.sqrt(total)
    scale = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    for t, to in zip(s["grads"], s["clipped"]):
        to.copy_(t.float() * scale)
    return [norm, *s["buckets"]]


def _plain_route(s, case):
    k, e = case["top_k"], case["experts"]
    logits = s["logits"].float()
    index = torch.arange(e, device="cuda", dtype=torch.int32)
    left, ids = logits.clone(), []
    for _ in range(k):
        best = left.max(dim=1, keepdim=True).values
        first = torch.where((left == best) & (left > -math.inf), index, e).min(dim=1).values
        ids.append(torch.where(first < e, first, -1))
        left = torch.where(index == first[:, None], -math.inf, left)
    ids = torch.stack(ids, 1).to(torch.int32)
    found = ids >= 0
    at = ids.clamp(min=0).long()
    top = logits.max(dim=1, keepdim=True).values
    top = torch.where(top > -math.inf, top, 0.0)
    raised = torch.exp(logits - top)
    chosen = torch.where(found, raised.gather(1, at), 0.0)
    below = (chosen if case["renormalize"] else raised).sum(dim=1, keepdim=True)
    below = torch.where(below > 0, below, 1.0)
    weights = chosen / below
    # Stable places by counting: earlier keys of the same expert, behind all smaller experts.
    flat = ids.flatten()
    hits = flat[:, None] == index
    rank = torch.cumsum(hits, 0, dtype=torch.int32)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(rank[-1], 0)
    to = flat.clamp(min=0).long()
    place = offsets[to] + rank.gather(1, to[:, None])[:, 0] - 1
    position = torch.where(flat >= 0, place, -1)
    order = torch.full((flat.numel() + 1,), -1, dtype=torch.int32, device="cuda")
    order[torch.where(flat >= 0, place, flat.numel()).long()] = torch.where(
        flat >= 0, torch.arange(flat.numel(), dtype=torch.int32, device="cuda"), -1)
    out = [ids, weights, offsets, order[:-1], position]
    if case["backward"]:
        inner = (weights * s["grad_weights"]).sum(dim=1, keepdim=True)
        grad = torch.where(found, weights * s["grad_weights"], 0.0)
        base = torch.zeros_like(logits)
        if case["renormalize"]:
            grad = grad - weights * inner
        else:
            base = -(raised / below) * inner
        out.append(base.scatter_add(1, at, grad).to(s["logits"].dtype))
    return out


def _plain_rows(s, case):
    if not case["gather"]:
        return None
    return torch.where(s["order"] < 0, 0, s["order"] // case["top_k"]).long()


def _plain_product(s, case):
    dtype = _DTYPES[case["dtype"]]
    at, rows, out = s["splits"], _plain_rows(s, case), []
    groups = [(i, at[i], at[i + 1]) for i in range(case["experts"]) if at[i + 1] > at[i]]
    n = s["order"].numel()

    def x_of(a, b):
        return (s["x"][a:b] if rows is None else s["x"][rows[a:b]]).float()

    if case["kind"] in ("forward", "step"):
        y = torch.zeros(n, case["outer"], dtype=dtype, device="cuda")
        for i, a, b in groups:
            y[a:b] = (x_of(a, b) @ s["weight"][i].float().t()).to(dtype)
        out.append(y)
    if case["kind"] in ("input_gradient", "step"):
        y = torch.zeros(n, case["inner"], dtype=dtype, device="cuda")
        for i, a, b in groups:
            y[a:b] = (s["dy"][a:b].float() @ s["weight"][i].float()).to(dtype)
        out.append(y)
    if case["kind"] in ("weight_gradient", "step"):
        y = torch.zeros(case["experts"], case["outer"], case["inner"], dtype=dtype, device="cuda")
        for i, a, b in groups:
            y[i] = (s["dy"][a:b].float().t() @ x_of(a, b)).to(dtype)
        out.append(y)
    return out


def _plain_combine(s, case):
    pos = s["position"].clamp(min=0).long()
    found = s["position"] >= 0
    z = s["z"]
    y = torch.zeros(case["tokens"], case["width"], device="cuda")
    for j in range(case["top_k"]):
        row = z[pos[:, j]].float()
        y = y + torch.where(found[:, j:j + 1], s["weights"][:, j:j + 1] * row, 0.0)
    out = [y.to(z.dtype)]
    if case["backward"]:
        dy = s["dy"].float()
        dz = torch.zeros(z.shape[0] + 1, case["width"], dtype=z.dtype, device="cuda")
        dw = torch.zeros_like(s["weights"])
        for j in range(case["top_k"]):
            dw[:, j] = torch.where(found[:, j], (dy * z[pos[:, j]].float()).sum(dim=1), 0.0)
            dz[torch.where(found[:, j], pos[:, j], z.shape[0])] = \
                (s["weights"][:, j:j + 1] * dy).to(z.dtype)
        out += [dz[:-1], dw]
    return out


# ---------------------------------------------------------------- work

def _rows(case):
    return case["tokens"] * case["top_k"] * (1.0 - case["padding"])


def work(case):
    if case["op"] == "route":
        t, e, n = case["tokens"], case["experts"], case["tokens"] * case["top_k"]
        size = _SIZE[case["dtype"]]
        total = t * e * size + 16 * n + 4 * (e + 1)
        if case["backward"]:
            total += t * e * size + 4 * n
        return dict(bytes=total, flops=t * e * (8 if case["backward"] else 4))
    if case["op"] == "product":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        n, rows = t * k, _rows(case)
        active = e * (1.0 - (1.0 - k / e) ** (t * (1.0 - case["padding"])))
        source = (t * (1.0 - case["padding"]) if case["gather"] else rows) * case["inner"] * 2
        matrix = case["inner"] * case["outer"] * 2
        index = 4 * (e + 1) + (4 * rows if case["gather"] else 0)
        parts = {"forward": source + active * matrix + n * case["outer"] * 2 + index,
                 "input_gradient": rows * case["outer"] * 2 + active * matrix
                 + n * case["inner"] * 2 + 4 * (e + 1),
                 "weight_gradient": rows * case["outer"] * 2 + source + e * matrix + index}
        flops = 2.0 * rows * case["inner"] * case["outer"]
        if case["kind"] == "step":      # the sources that two products share are read once
            total = sum(parts.values()) - active * matrix - source - rows * case["outer"] * 2 \
                - 4 * (e + 1) - index
            return dict(bytes=int(total), flops=int(3 * flops))
        return dict(bytes=int(parts[case["kind"]]), flops=int(flops))
    if case["op"] == "combine":
        t, n, rows = case["tokens"], case["tokens"] * case["top_k"], _rows(case)
        row = case["width"] * _SIZE[case["dtype"]]
        total, flops = rows * row + t * row + 8 * n, 2 * rows * case["width"]
        if case["backward"]:
            total += t * row + n * row + 4 * n
            flops += 3 * rows * case["width"]
        return dict(bytes=int(total), flops=int(flops))
    total = sum(2 * size * _SIZE[d] for size, d in zip(_clip_shapes(case), _clip_dtypes(case)))
    return dict(bytes=total, flops=3 * sum(_clip_shapes(case)))


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "product": _exact_product, "combine": _exact_combine,
            "clip": _exact_clip}[case["op"]](s, case)


def _exact_route(s, case):
    k, e = case["top_k"], case["experts"]
    x = s["logits"].double().cpu()
    best = torch.sort(x, dim=1, descending=True, stable=True)
    ok = best.values[:, :k] > -math.inf
    ids = torch.where(ok, best.indices[:, :k], -1)
    p = torch.nan_to_num(torch.softmax(x, dim=1), nan=0.0)
    weights = torch.where(ok, p.gather(1, ids.clamp(min=0)), 0.0)
    if case["renormalize"]:
        weights = torch.nan_to_num(weights / weights.sum(1, keepdim=True), nan=0.0)
    key = torch.where(ids < 0, e, ids).flatten()
    order = torch.sort(key, stable=True).indices
    offsets = torch.searchsorted(key[order], torch.arange(e + 1))
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel())
    position[key == e] = -1
    order = torch.where(torch.arange(order.numel()) < offsets[-1], order, -1)
    out = [ids.int(), weights, offsets.int(), order.int(), position.int()]
    if case["backward"]:
        dw = s["grad_weights"].double().cpu()
        dot = (weights * dw).sum(1, keepdim=True)
        full = torch.zeros_like(x)
        if case["renormalize"]:
            full.scatter_add_(1, ids.clamp(min=0), weights * (dw - dot))
        else:
            full.scatter_add_(1, ids.clamp(min=0), weights * dw)
            full -= p * dot
        out.append(full)
    return out


def _exact_product(s, case):
    if case["kind"] != "step":
        flops = work(case)["flops"]
    else:
        flops = work(case)["flops"] / 3
    if flops > 4e12:
        return None
    at, e, n = s["splits"], case["experts"], s["order"].numel()
    source = s["order"].long() // case["top_k"] if case["gather"] else \
        torch.arange(n, device="cuda")
    out = []
    if case["kind"] in ("forward", "step"):
        y = torch.zeros(n, case["outer"], dtype=torch.float64, device="cuda")
        for i in range(e):
            y[at[i]:at[i + 1]] = torch.einsum(
                "mk,nk->mn", s["x"].index_select(0, source[at[i]:at[i + 1]]).double(),
                s["weight"][i].double())
        out.append(y)
    if case["kind"] in ("input_gradient", "step"):
        y = torch.zeros(n, case["inner"], dtype=torch.float64, device="cuda")
        for i in range(e):
            y[at[i]:at[i + 1]] = torch.einsum("mn,nk->mk", s["dy"][at[i]:at[i + 1]].double(),
                                              s["weight"][i].double())
        out.append(y)
    if case["kind"] in ("weight_gradient", "step"):
        y = torch.zeros(e, case["outer"], case["inner"], dtype=torch.float64, device="cuda")
        for i in range(e):
            y[i] = torch.einsum("mn,mk->nk", s["dy"][at[i]:at[i + 1]].double(),
                                s["x"].index_select(0, source[at[i]:at[i + 1]]).double())
        out.append(y)
    return out


def _exact_combine(s, case):
    z, w, pos = s["z"].double(), s["weights"].double(), s["position"].long()
    z = torch.cat([z, torch.zeros(1, case["width"], dtype=z.dtype, device="cuda")])  # row -1 is zero
    y = torch.zeros(case["tokens"], case["width"], dtype=z.dtype, device="cuda")
    for j in range(case["top_k"]):
        y += w[:, j, None] * z[pos[:, j]]
    out = [y]
    if case["backward"]:
        dy = s["dy"].double()
        dz, dw = torch.zeros_like(z), torch.zeros_like(w)
        for j in range(case["top_k"]):
            keep = pos[:, j] >= 0
            dz[pos[keep, j]] = w[keep, j, None] * dy[keep]
            dw[:, j] = torch.einsum("td,td->t", dy, z[pos[:, j]])
        out += [dz[:-1], dw]
    return out


def _exact_clip(s, case):
    norm = math.sqrt(math.fsum(float(torch.sum(t.double() ** 2)) for t in s["grads"]))
    scale = min(1.0, s["max_norm"] / (norm + 1e-6))
    out = []
    for dtype in dict.fromkeys(t.dtype for t in s["grads"]):
        parts = [torch.nn.functional.pad(t.double() * scale, (0, -t.numel() % 64))
                 for t in s["grads"] if t.dtype == dtype]
        out.append(torch.cat(parts))
    return [torch.tensor(norm, dtype=torch.float64), *out]
