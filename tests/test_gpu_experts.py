"""The expert-layer operators on the GPU against plain 64-bit forms.

Tolerances follow from the arithmetic.  A value rounded once to a type with
unit roundoff u is off by at most u of itself; a sum of m terms in 32 bits
loses at most one unit in the last place (2^-23) of the sum of magnitudes per
addition; float16 results below its normal range are off by at most 2^-25.
"""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import cluster_distributed_shared_gb300 as dh  # noqa: E402

pytestmark = pytest.mark.gpu

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -23}
FLOOR = {torch.bfloat16: 2.0 ** -130, torch.float16: 2.0 ** -24, torch.float32: 2.0 ** -130}


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()


def generator(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def close(got, want, magnitude, terms):
    """|got - want| within rounding to got's type and `terms` 32-bit additions
    of terms whose magnitudes sum to `magnitude`."""
    assert got.shape == want.shape
    g = got.detach().cpu().double()
    bound = UNIT[got.dtype] * want.abs() + terms * 2.0 ** -23 * magnitude + FLOOR[got.dtype]
    bad = ~((g - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} differ, first {bad.nonzero()[0].tolist()}"


# ------------------------------------------------------------------- route

def route_exact(logits, k, renormalize):
    x = logits.double().cpu()
    x = torch.where(x.isnan(), -math.inf, x)
    best = torch.sort(x, dim=1, descending=True, stable=True)
    ok = best.values[:, :k] > -math.inf
    ids = torch.where(ok, best.indices[:, :k], -1)
    top = x.max(dim=1, keepdim=True).values
    p = torch.where(x == math.inf, 1.0, torch.where(top == math.inf, 0.0, torch.exp(x - top)))
    p = torch.where(x > -math.inf, p, 0.0)
    w = torch.where(ok, p.gather(1, ids.clamp(min=0)), 0.0)
    below = (w if renormalize else p).sum(1, keepdim=True)
    below = torch.where(below > 0, below, 1.0)
    return ids.int(), w / below, p / below


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,experts,k", [(1, 1, 1), (1, 64, 4), (5, 33, 32), (130, 60, 3),
                                              (257, 256, 8), (9, 257, 2), (33, 1024, 6)])
def test_route_and_gradient(tokens, experts, k, dtype, renormalize):
    g = generator(tokens * 1000 + experts)
    logits = torch.randn(tokens, experts, generator=g).to(dtype)
    logits[:, torch.rand(experts, generator=g) < 0.1] = -math.inf
    logits[0, experts // 2] = math.nan
    if tokens > 4:
        logits[1] = -math.inf          # nothing to choose
        logits[2] = 0.25               # all equal: the lowest indexes
        logits[3, experts - 1] = math.inf
        logits[4, ::2] = 0.0
        logits[4, 1::2] = -0.0         # equal to +0
    wide = torch.zeros(tokens, experts + 3, dtype=dtype)
    wide[:, :experts] = logits
    dev = wide.cuda()[:, :experts]     # rows with a stride
    ids, w = dh.dsmem_route(dev, k, renormalize=renormalize)
    want_ids, want_w, p = route_exact(logits, k, renormalize)
    assert torch.equal(ids.cpu(), want_ids)
    # expf is within 2 units, the argument's rounding within |x - top| units,
    # the sum adds one unit for each of at most 37 levels, the division one
    assert (w.cpu().double() - want_w).abs().max() <= 64 * 2.0 ** -24
    dw = torch.randn(tokens, k, generator=g)
    got = dh.dsmem_route_backward(dev, ids, w, dw.cuda(), renormalize=renormalize)
    d = dw.double()
    dot = torch.where(want_ids >= 0, want_w * d, 0.0).sum(1, keepdim=True)
    full = torch.zeros(tokens, experts, dtype=torch.float64)
    part = want_w * (d - dot) if renormalize else want_w * d
    full.scatter_add_(1, want_ids.clamp(min=0).long(), torch.where(want_ids >= 0, part, 0.0))
    if not renormalize:
        full -= p * dot
    bound = UNIT[dtype] * full.abs() + 128 * 2.0 ** -24 * (d.abs().max() + 1) + FLOOR[dtype]
    assert ((got.cpu().double() - full).abs() <= bound).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_route_with_masks_of_the_lowest_value(dtype):
    """The type's lowest value is a number: chosen after all others, with no
    weight beside them, and an even share where it is all there is."""
    low = torch.finfo(dtype).min
    logits = torch.full((3, 40), low, dtype=dtype)
    logits[0, 7], logits[0, 31] = 1.0, 2.0
    logits[2, :38] = -math.inf
    ids, w = dh.dsmem_route(logits.cuda(), 3)
    assert ids.tolist() == [[31, 7, 0], [0, 1, 2], [38, 39, -1]]
    want = torch.tensor([[1 / (1 + math.exp(-1)), 1 / (1 + math.exp(1)), 0], [1 / 3] * 3, [0.5, 0.5, 0]])
    assert (w.cpu() - want).abs().max() <= 2.0 ** -22
    grad = dh.dsmem_route_backward(logits.cuda(), ids, w, torch.ones(3, 3).cuda())
    assert torch.isfinite(grad).all() and grad.abs().max() <= 2.0 ** -20   # equal gradients cancel


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_against_differences(renormalize):
    g = generator(3)
    logits = torch.randn(4, 12, generator=g).double()
    dw = torch.randn(4, 3, generator=g)
    dev = logits.float().cuda()
    ids, w = dh.dsmem_route(dev, 3, renormalize=renormalize)
    grad = dh.dsmem_route_backward(dev, ids, w, dw.cuda(), renormalize=renormalize).cpu().double()
    base, step = dev.cpu().double(), 1e-6

    def value(x):
        p = torch.softmax(x, 1).gather(1, ids.cpu().long())
        if renormalize:
            p = p / p.sum(1, keepdim=True)
        return (p * dw.double()).sum()

    for t in range(4):
        for e in range(12):
            up, down = base.clone(), base.clone()
            up[t, e] += step
            down[t, e] -= step
            slope = (value(up) - value(down)) / (2 * step)
            assert abs(float(slope) - float(grad[t, e])) <= 1e-5


# ------------------------------------------------------------------- group

def group_exact(keys, groups):
    key = torch.where((keys < 0) | (keys >= groups), groups, keys).long()
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=groups + 1)[:groups]
    offsets = torch.zeros(groups + 1, dtype=torch.long)
    offsets[1:] = counts.cumsum(0)
    position = torch.empty_like(order)
    position[order] = torch.arange(len(keys))
    position[key == groups] = -1
    order = torch.where(torch.arange(len(keys)) < offsets[-1], order, -1)
    return offsets.int(), order.int(), position.int()


@pytest.mark.parametrize("n,groups", [(0, 5), (1, 1), (1, 7), (31, 3), (32, 32), (33, 64), (1000, 257),
                                      (4097, 8), (70001, 60), (131072, 256), (300000, 1024),
                                      (50000, 5000), (40000, 32768), (262145, 77), (1000003, 256),
                                      (700000, 5000), (300001, 20000)])
@pytest.mark.parametrize("kind", ["uniform", "skewed", "one", "dropped"])
def test_group(n, groups, kind):
    g = generator(n + groups)
    keys = torch.randint(0, groups, (n,), generator=g, dtype=torch.int32)
    if kind == "skewed":
        keys = (keys.float() ** 2 / groups).to(torch.int32)
        keys[torch.rand(n, generator=g) < 0.1] = -1
        keys[torch.rand(n, generator=g) < 0.05] = groups
    if kind == "one":
        keys[:] = groups - 1
    if kind == "dropped":
        keys[:] = -2 ** 31
    got = dh.dsmem_group(keys.cuda(), groups)
    for a, b in zip(got, group_exact(keys, groups)):
        assert torch.equal(a.cpu(), b)


def test_group_counts_are_the_histogram():
    keys = torch.randint(-3, 300, (100003,), generator=generator(1), dtype=torch.int32).cuda()
    offsets = dh.dsmem_group(keys, 256)[0]
    assert torch.equal(offsets[1:] - offsets[:-1], dh.dsmem_hist(keys, 256))


# ---------------------------------------------------------------- products

def routing(g, tokens, experts, k, skew, drop):
    """Offsets, order and n of a routing with empty groups where skewed."""
    score = skew * torch.randn(experts, generator=g) * 2 + torch.rand(tokens, experts, generator=g)
    ids = score.topk(k, dim=1).indices.int()
    ids[torch.rand(tokens, generator=g) < drop] = -1
    return group_exact(ids.flatten(), experts)


PRODUCTS = [
    # tokens, experts, k, inner, outer, skew
    (1, 8, 2, 64, 128, 0.0),
    (1, 4, 1, 512, 72, 0.0),
    (3, 5, 1, 8, 8, 0.0),
    (17, 4, 2, 200, 136, 0.0),
    (40, 3, 1, 1003, 517, 0.0),
    (64, 16, 4, 320, 264, 1.0),
    (129, 2, 1, 72, 520, 0.0),
    (300, 7, 3, 129, 65, 1.0),
    (515, 3, 2, 328, 256, 0.0),
    (1100, 4, 2, 136, 392, 0.5),
    (2, 300, 2, 136, 64, 0.0),
    # one group, few rows or few channels: the depth is split over a cluster
    (1, 1, 1, 4096, 256, 0.0),
    (3, 2, 2, 1032, 1032, 0.0),
    (40, 1, 1, 1024, 136, 0.0),
    (60, 2, 1, 264, 2048, 0.0),
    (2100, 1, 1, 64, 128, 0.0),
    # enough tiles for pairs of CTAs, 128 and 256 rows wide
    (1300, 16, 1, 520, 800, 0.5),
    (3000, 4, 1, 776, 1304, 0.5),
    (2500, 5, 2, 1100, 1001, 1.0),
    (700, 30, 1, 520, 264, 0.0),
    # many rows of few channels
    (9900, 3, 1, 72, 104, 0.5),
]


def product_inputs(case, dtype, gather, drop=0.05):
    tokens, experts, k, inner, outer, skew = case
    g = generator(tokens + inner)
    offsets, order, _ = routing(g, tokens, experts, k, skew, drop if tokens > 8 else 0.0)
    n, rows = tokens * k, tokens if gather else tokens * k
    x = torch.randn(rows, inner, generator=g).to(dtype)
    w = (torch.randn(experts, outer, inner, generator=g) / math.sqrt(inner)).to(dtype)
    dy = torch.randn(n, outer, generator=g).to(dtype)
    source = torch.where(order < 0, 0, order // k).long() if gather else torch.arange(n)
    end = int(offsets[-1])
    dy[end:] = math.nan                       # places of no group are not read
    if gather:
        used = torch.zeros(rows, dtype=torch.bool)
        used[source[:end]] = True
        x[~used] = math.nan                   # nor are rows that no place names
    else:
        x[end:] = math.nan
    rows_of = dict(order=order.cuda(), fan=k) if gather else {}
    return x, w, dy, offsets, source, rows_of


def spans(offsets):
    at = offsets.tolist()
    return [(g, a, b) for g, (a, b) in enumerate(zip(at, at[1:])) if b > a]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("case", PRODUCTS)
def test_products(case, gather, dtype):
    x, w, dy, offsets, source, rows_of = product_inputs(case, dtype, gather)
    n, outer, inner = dy.shape[0], dy.shape[1], x.shape[1]
    y = torch.zeros(n, outer, dtype=torch.float64)
    my = torch.zeros_like(y)
    dx = torch.zeros(n, inner, dtype=torch.float64)
    mdx = torch.zeros_like(dx)
    dw = torch.zeros(w.shape, dtype=torch.float64)
    mdw = torch.zeros_like(dw)
    xd, wd, dyd = x.double(), w.double(), dy.double()
    for e, a, b in spans(offsets):
        rows = xd[source[a:b]]
        y[a:b], my[a:b] = rows @ wd[e].T, rows.abs() @ wd[e].abs().T
        dx[a:b], mdx[a:b] = dyd[a:b] @ wd[e], dyd[a:b].abs() @ wd[e].abs()
        dw[e], mdw[e] = dyd[a:b].T @ rows, dyd[a:b].abs().T @ rows.abs()
    off = offsets.cuda()
    for out_dtype in (dtype, torch.float32):
        got = dh.dsmem_grouped_matmul(x.cuda(), w.cuda(), off, out_dtype=out_dtype, **rows_of)
        close(got, y, my, inner)
        got = dh.dsmem_grouped_matmul(dy.cuda(), w.cuda(), off, transpose=True, out_dtype=out_dtype)
        close(got, dx, mdx, outer)
        got = dh.dsmem_grouped_matmul_wgrad(dy.cuda(), x.cuda(), off, out_dtype=out_dtype, **rows_of)
        close(got, dw, mdw, n)


@pytest.mark.parametrize("case", [PRODUCTS[3], PRODUCTS[5], PRODUCTS[8]])
def test_products_of_views(case):
    """Row and group strides, and bases 2 bytes off alignment."""
    x, w, dy, offsets, source, rows_of = product_inputs(case, torch.bfloat16, True)
    off = offsets.cuda()

    def view(t, pad, shift):
        buf = torch.full((t.numel() // t.shape[-1], t.shape[-1] + pad), math.nan, dtype=t.dtype)
        buf[:, shift:shift + t.shape[-1]] = t.reshape(-1, t.shape[-1])
        return buf.cuda().view(*t.shape[:-1], -1)[..., shift:shift + t.shape[-1]]

    want = (dh.dsmem_grouped_matmul(x.cuda(), w.cuda(), off, **rows_of),
            dh.dsmem_grouped_matmul(dy.cuda(), w.cuda(), off, transpose=True),
            dh.dsmem_grouped_matmul_wgrad(dy.cuda(), x.cuda(), off, **rows_of))
    for pad, shift in [(8, 0), (16, 8), (8, 1), (3, 2)]:
        vx, vw, vdy = view(x, pad, shift), view(w, pad, shift), view(dy, pad, shift)
        got = (dh.dsmem_grouped_matmul(vx, vw, off, **rows_of),
               dh.dsmem_grouped_matmul(vdy, vw, off, transpose=True),
               dh.dsmem_grouped_matmul_wgrad(vdy, vx, off, **rows_of))
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_products_without_rows():
    dev = dict(device="cuda", dtype=torch.bfloat16)
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    w = torch.randn(4, 24, 16, **dev)
    assert dh.dsmem_grouped_matmul(torch.empty(0, 16, **dev), w, off).shape == (0, 24)
    dw = dh.dsmem_grouped_matmul_wgrad(torch.empty(0, 24, **dev), torch.empty(0, 16, **dev), off)
    assert dw.shape == (4, 24, 16) and not dw.any()
    # rows, but all of no group
    y = dh.dsmem_grouped_matmul(torch.full((9, 16), math.nan, **dev), w, off)
    assert y.shape == (9, 24) and not y.any()
    # an order that names rows outside x gives zeros
    order = torch.tensor([0, 7, -1, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 0, 4, 4, 4], dtype=torch.int32, device="cuda")
    x = torch.randn(2, 16, **dev)
    y = dh.dsmem_grouped_matmul(x, w, off, order=order)
    assert y[0].any() and not y[1:].any()
    dw = dh.dsmem_grouped_matmul_wgrad(torch.ones(4, 24, **dev), x, off, order=order)
    assert torch.equal(dw[1], x[:1].expand(24, 16))


def test_products_with_offsets_out_of_range_stay_inside():
    dev = dict(device="cuda", dtype=torch.float16)
    x, w = torch.ones(40, 64, **dev), torch.ones(3, 128, 64, **dev)
    dy = torch.ones(40, 128, **dev)
    for off in ([0, -5, 2 ** 31 - 1, 7], [3, 30, 10, 20], [-1, -1, -1, -1]):
        t = torch.tensor(off, dtype=torch.int32, device="cuda")
        assert dh.dsmem_grouped_matmul(x, w, t).shape == (40, 128)
        assert dh.dsmem_grouped_matmul(dy, w, t, transpose=True).shape == (40, 64)
        assert dh.dsmem_grouped_matmul_wgrad(dy, x, t).shape == (3, 128, 64)
        torch.cuda.synchronize()


def test_products_are_repeatable_and_ordered_by_stream():
    case = PRODUCTS[8]
    x, w, dy, offsets, source, rows_of = product_inputs(case, torch.bfloat16, True)
    args = (x.cuda(), w.cuda(), offsets.cuda())
    want = dh.dsmem_grouped_matmul(*args, **rows_of)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = dh.dsmem_grouped_matmul(*args, stream=side, **rows_of)
        side.synchronize()
        assert torch.equal(got, want)


# ----------------------------------------------------------------- combine

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("tokens,k,width", [(1, 1, 1), (1, 4, 2048), (7, 3, 129), (33, 8, 264), (50, 2, 4100),
                                            (300, 5, 72)])
def test_combine_and_gradients(tokens, k, width, dtype):
    g = generator(tokens + width)
    ids = torch.randint(0, 9, (tokens, k), generator=g, dtype=torch.int32)
    if tokens > 1:
        ids[torch.rand(tokens, k, generator=g) < 0.2] = -1
        ids[0] = -1                                     # a token without any row
    offsets, order, position = group_exact(ids.flatten(), 9)
    position = position.view(tokens, k)
    end = int(offsets[-1])
    z = torch.randn(tokens * k, width, generator=g).to(dtype)
    z[end:] = math.nan
    dy = torch.randn(tokens, width, generator=g).to(dtype)
    w = torch.rand(tokens, k, generator=g)
    w[position < 0] = math.nan                          # weights of dropped rows are not read
    ok = position >= 0
    wd = torch.where(ok, w.double(), 0.0)
    rows = torch.where(ok[..., None], z.double()[position.clamp(min=0).long()], 0.0)
    dev = [t.cuda() for t in (z, position, w)]
    close(dh.dsmem_combine(*dev), (wd[..., None] * rows).sum(1), (wd[..., None] * rows).abs().sum(1), k + 1)
    close(dh.dsmem_combine(*dev[:2]), rows.sum(1), rows.abs().sum(1), k)
    dz, dw = dh.dsmem_combine_backward(dy.cuda(), dev[0], dev[1], order.cuda(), dev[2])
    want = torch.zeros(tokens * k, width, dtype=torch.float64)
    want[position[ok].long()] = (wd[..., None] * dy.double()[:, None, :])[ok]
    close(dz, want, want.abs(), 1)
    prod = rows * dy.double()[:, None, :]
    close(dw, prod.sum(-1), prod.abs().sum(-1), width)
    strided = torch.randn(tokens * k, width + 5, generator=g).to(dtype).cuda()[:, 1:width + 1]
    a = dh.dsmem_combine(strided, dev[1])
    assert torch.equal(a, dh.dsmem_combine(strided.contiguous(), dev[1]))


def test_combine_gradients_against_differences():
    g = generator(5)
    tokens, k, width = 5, 3, 6
    ids = torch.randint(0, 4, (tokens, k), generator=g, dtype=torch.int32)
    ids[1, 2] = -1
    offsets, order, position = group_exact(ids.flatten(), 4)
    position = position.view(tokens, k)
    z = torch.randn(tokens * k, width, generator=g)
    w, dy = torch.rand(tokens, k, generator=g), torch.randn(tokens, width, generator=g)
    dz, dw = dh.dsmem_combine_backward(dy.cuda(), z.cuda(), position.cuda(), order.cuda(), w.cuda())

    def value(zz, ww):
        rows = torch.where((position >= 0)[..., None], zz[position.clamp(min=0).long()], 0.0)
        return float(((ww[..., None] * rows).sum(1) * dy.double()).sum())

    # the function is linear in each, so a difference over a step of 1 is exact
    for t, grad in ((0, dz), (1, dw)):
        args = [z.double(), w.double()]
        base = value(*args)
        flat = grad.cpu().flatten()
        for i in range(flat.numel()):
            moved = [a.clone() for a in args]
            moved[t].view(-1)[i] += 1.0
            assert abs(value(*moved) - base - float(flat[i])) <= 1e-5


# -------------------------------------------------------------------- clip

@pytest.mark.parametrize("sizes", [[1], [0, 3, 0], [8192], [8193, 1, 7, 100000, 31], [5] * 2100,
                                   [3_000_001, 64]])
@pytest.mark.parametrize("max_norm", [1.0, 1e9])
def test_clip(sizes, max_norm):
    g = generator(len(sizes))
    types = [torch.float32, torch.bfloat16, torch.float16]
    grads = [torch.randn(n, generator=g).to(types[i % 3]) for i, n in enumerate(sizes)]
    total = math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in grads))
    scale = min(1.0, max_norm / (total + 1e-6))
    dev = [t.cuda() for t in grads]
    out = [torch.full_like(t, math.nan) for t in dev]
    norm = dh.dsmem_grad_clip(dev, max_norm, out=out)
    # 32 squares a thread in 32 bits, the rest in 64
    assert abs(float(norm) - total) <= 34 * 2.0 ** -24 * total + 2.0 ** -24 * total
    for a, b, t in zip(out, grads, dev):
        want = b.double() * scale
        close(a, want, want.abs(), 36)
        assert torch.equal(t.cpu(), b)
    assert torch.equal(dh.dsmem_grad_clip(dev, max_norm), norm)       # in place
    for a, b in zip(out, dev):
        assert torch.equal(a, b)


def test_clip_of_views_and_extremes():
    base = torch.randn(10001, generator=generator(2)).cuda()
    views = [base[1:4000], base[4001:10000]]
    out = [torch.empty(3999, device="cuda"), torch.empty(6001, device="cuda")[2:]]
    norm = dh.dsmem_grad_clip(views, 1.0, out=out)
    want = math.sqrt(sum(float((v.double() ** 2).sum()) for v in views))
    assert abs(float(norm) - want) <= 36 * 2.0 ** -24 * want
    for scale in (1e30, 1e-30):                       # squares outside 32 bits
        big = [torch.full((1000,), scale, device="cuda"), torch.full((24,), scale, device="cuda")]
        norm = dh.dsmem_grad_clip(big, 1.0)
        assert abs(float(norm) / (scale * 32.0) - 1) <= 1e-6
        assert abs(float(big[0][0]) - min(scale, 1 / 32)) <= 1e-6 * min(scale, 1 / 32)
    zero = [torch.zeros(70000, device="cuda", dtype=torch.bfloat16)]
    assert float(dh.dsmem_grad_clip(zero, 1.0)) == 0.0 and not zero[0].any()
    inf = [torch.tensor([1.0, math.inf, 2.0], device="cuda")]
    assert float(dh.dsmem_grad_clip(inf, 1.0)) == math.inf
    assert inf[0][0] == 0 and inf[0][1].isnan() and inf[0][2] == 0
    nan = [torch.tensor([1.0, math.nan], device="cuda"), torch.ones(3, device="cuda")]
    assert dh.dsmem_grad_clip(nan, 1.0).isnan() and nan[1].isnan().all()
    assert float(dh.dsmem_grad_clip([], 1.0)) == 0.0


# Runs long enough that CTAs share their pieces, in lists of one table and of
# two (the second with short runs), beside sizes that end inside a chunk.
@pytest.mark.parametrize("count,size", [(3, 83_000_011), (1300, 300_007)])
def test_clip_of_long_runs(count, size):
    g = torch.Generator(device="cuda").manual_seed(count)
    flat = torch.randn(count * (size + 5), generator=g, device="cuda", dtype=torch.bfloat16)
    grads = [flat[i * (size + 5):i * (size + 5) + size] for i in range(count)]
    kept = flat.clone()
    out = torch.full_like(flat, math.nan)
    clipped = [out[i * (size + 5):i * (size + 5) + size] for i in range(count)]
    total = math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in grads))
    norm = dh.dsmem_grad_clip(grads, 2.0, out=clipped)
    assert abs(float(norm) - total) <= 35 * 2.0 ** -24 * total
    assert torch.equal(flat, kept)
    assert torch.equal(dh.dsmem_grad_clip(grads, 2.0), norm)          # in place
    for i in range(count):
        want = kept[i * (size + 5):i * (size + 5) + size].double() * (2.0 / (total + 1e-6))
        # the factor: 35 steps of 2^-24 of the norm and one of its own; one of the product, and bf16
        assert ((clipped[i].double() - want).abs() <= want.abs() * (2.0 ** -8 + 37 * 2.0 ** -24)).all()
        assert torch.equal(clipped[i], grads[i])
    gaps = out.view(count, size + 5)[:, size:]
    assert gaps.isnan().all() and torch.equal(flat.view(count, size + 5)[:, size:],
                                              kept.view(count, size + 5)[:, size:])


# ---------------------------------------------------------------- refusals

def test_refusals():
    f = torch.randn(8, 16, device="cuda")
    h = f.to(torch.bfloat16)
    i = torch.zeros(8, dtype=torch.int32, device="cuda")
    w = torch.randn(2, 4, 16, device="cuda", dtype=torch.bfloat16)
    off = torch.tensor([0, 4, 8], dtype=torch.int32, device="cuda")
    for call, error in [
        (lambda: dh.dsmem_route(f.cpu(), 2), TypeError),
        (lambda: dh.dsmem_route(f.double(), 2), TypeError),
        (lambda: dh.dsmem_route(f.t(), 2), ValueError),
        (lambda: dh.dsmem_route(f, 17), dh.DsmemHistError),
        (lambda: dh.dsmem_route(f, 0), dh.DsmemHistError),
        (lambda: dh.dsmem_route(torch.zeros(2, 1025, device="cuda"), 2), dh.DsmemHistError),
        (lambda: dh.dsmem_group(i.long(), 4), TypeError),
        (lambda: dh.dsmem_group(i[::2], 4), ValueError),
        (lambda: dh.dsmem_group(i, 0), dh.DsmemHistError),
        (lambda: dh.dsmem_group(i, 32769), dh.DsmemHistError),
        (lambda: dh.dsmem_grouped_matmul(f, w.float(), off), TypeError),
        (lambda: dh.dsmem_grouped_matmul(h, w.half(), off), TypeError),
        (lambda: dh.dsmem_grouped_matmul(h[:, :8], w, off), ValueError),
        (lambda: dh.dsmem_grouped_matmul(h, w, off[:2]), ValueError),
        (lambda: dh.dsmem_grouped_matmul(h, w, off, out_dtype=torch.float16), TypeError),
        (lambda: dh.dsmem_grouped_matmul(h, w, off, fan=0), dh.DsmemHistError),
        (lambda: dh.dsmem_grouped_matmul(h, w.transpose(1, 2), off), ValueError),
        (lambda: dh.dsmem_grouped_matmul_wgrad(h, h[:7], off), ValueError),
        (lambda: dh.dsmem_combine(f, i), ValueError),
        (lambda: dh.dsmem_combine(f, i.view(4, 2), torch.ones(2, 4, device="cuda")), ValueError),
        (lambda: dh.dsmem_combine_backward(f[:4], f, i.view(4, 2), i, None), TypeError),
        (lambda: dh.dsmem_grad_clip([f, f.cpu()], 1.0), TypeError),
        (lambda: dh.dsmem_grad_clip([f], 1.0, out=[h]), ValueError),
        (lambda: dh.dsmem_grad_clip([f], 0.0), dh.DsmemHistError),
        (lambda: dh.dsmem_grad_clip([f], math.nan), dh.DsmemHistError),
    ]:
        with pytest.raises(error):
            call()


def test_offsets_past_32_bits():
    """Outputs and inputs of more than 2^31 elements, looked at near their ends."""
    g = generator(8)
    n, inner, outer = 70001, 16, 32768
    x = torch.randn(n, inner, generator=g).to(torch.bfloat16)
    w = torch.randn(2, outer, inner, generator=g).to(torch.bfloat16)
    off = torch.tensor([0, 30000, n], dtype=torch.int32, device="cuda")
    y = dh.dsmem_grouped_matmul(x.cuda(), w.cuda(), off)
    xd, wd = x[-3:].double(), w[1].double()
    close(y[-3:], xd @ wd.T, xd.abs() @ wd.abs().T, inner)
    position = torch.tensor([[n - 1, n - 2], [n - 3, -1]], dtype=torch.int32, device="cuda")
    z = dh.dsmem_combine(y, position).cpu().double()
    last = y[-3:].cpu().double()
    want = torch.stack([last[2] + last[1], last[0]])
    assert ((z - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -22 * last.abs().sum(0)).all()
    # the same rows as a source
    dx = dh.dsmem_grouped_matmul(y, w.cuda(), off, transpose=True)[-3:]
    close(dx, last @ wd, last.abs() @ wd.abs(), outer)
    del y
    groups, inner, outer = 70, 4096, 8192
    x, dy = (torch.randn(groups, c, generator=g).to(torch.bfloat16) for c in (inner, outer))
    off = torch.arange(groups + 1, dtype=torch.int32, device="cuda")
    dw = dh.dsmem_grouped_matmul_wgrad(dy.cuda(), x.cuda(), off)
    want = dy[-1].double()[:, None] * x[-1].double()[None]
    close(dw[-1], want, want.abs(), 1)
    del dw
    count = 2 ** 31 + 5
    grad = torch.full((count,), 2.0 ** -10, dtype=torch.bfloat16, device="cuda")
    norm = dh.dsmem_grad_clip([grad], 1.0)
    want = 2.0 ** -10 * math.sqrt(count)
    assert abs(float(norm) - want) <= 1e-6 * want
    ends = torch.stack([grad[0], grad[2 ** 31 - 1], grad[-1]]).double().cpu()
    assert ((ends - 2.0 ** -10 / want).abs() <= 2.0 ** -8 * 2.0 ** -10 / want).all()


def test_every_operator_on_a_given_stream():
    """With `stream`, outputs belong to it and equal the current stream's."""
    g = generator(11)
    logits = torch.randn(300, 24, generator=g).cuda()
    x = torch.randn(300, 64, generator=g).to(torch.bfloat16).cuda()
    up = torch.randn(24, 128, 64, generator=g).to(torch.bfloat16).cuda()

    def layer(**on):
        ids, w = dh.dsmem_route(logits, 3, **on)
        off, order, pos = dh.dsmem_group(ids, 24, **on)
        pos = pos.view(300, 3)
        h = dh.dsmem_grouped_matmul(x, up, off, order=order, fan=3, **on)
        y = dh.dsmem_combine(h, pos, w, **on)
        dz, dw = dh.dsmem_combine_backward(y, h, pos, order, w, **on)
        dx = dh.dsmem_grouped_matmul(dz, up, off, transpose=True, **on)
        dup = dh.dsmem_grouped_matmul_wgrad(dz, x, off, order=order, fan=3, **on)
        dl = dh.dsmem_route_backward(logits, ids, w, dw, **on)
        norm = dh.dsmem_grad_clip([dup, dl], 1.0, **on)
        return [ids, w, off, order, pos, h, y, dz, dw, dx, dup, dl, norm]

    want = layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = layer(stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_a_failed_scratch_allocation_is_reported(monkeypatch):
    f = [torch.ones(8, device="cuda")]
    monkeypatch.setenv("DSMEM_HIST_TEST_FAIL_ALLOC", "1")
    with pytest.raises(dh.DsmemHistError) as e:
        dh.dsmem_grad_clip(f, 1.0)
    assert e.value.code == dh.DSMEM_HIST_ENOMEM
    monkeypatch.delenv("DSMEM_HIST_TEST_FAIL_ALLOC")
    assert float(dh.dsmem_grad_clip(f, 1e9)) == pytest.approx(math.sqrt(8), rel=1e-6)


@pytest.mark.parametrize("case", [PRODUCTS[0], PRODUCTS[11], PRODUCTS[16], PRODUCTS[17]])
def test_a_wait_that_gives_up_is_reported_by_the_next_call(case, monkeypatch):
    """The copies of the last stage are withheld, so the wait for them runs
    out with nothing of it in flight (a solo, a split and two paired shapes)."""
    x, w, dy, offsets, source, rows_of = product_inputs(case, torch.bfloat16, True)
    args = (x.cuda(), w.cuda(), offsets.cuda())
    want = dh.dsmem_grouped_matmul(*args, **rows_of)
    torch.cuda.synchronize()
    monkeypatch.setenv("DSMEM_HIST_TEST_WAIT_CYCLES", "200000")
    monkeypatch.setenv("DSMEM_HIST_TEST_WITHHOLD_LAST_ROUND", "1")
    dh.dsmem_grouped_matmul(*args, **rows_of)
    torch.cuda.synchronize()
    monkeypatch.delenv("DSMEM_HIST_TEST_WAIT_CYCLES")
    monkeypatch.delenv("DSMEM_HIST_TEST_WITHHOLD_LAST_ROUND")
    with pytest.raises(dh.DsmemHistError) as e:
        dh.dsmem_grouped_matmul(*args, **rows_of)
    assert e.value.code == dh.DSMEM_HIST_ETIMEOUT and "grouped product" in str(e.value)
    assert dh.dsmem_hist_device_status() == 2 and dh.dsmem_hist_device_status() == 0
    assert torch.equal(dh.dsmem_grouped_matmul(*args, **rows_of), want)
