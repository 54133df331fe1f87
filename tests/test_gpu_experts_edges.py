"""The expert-layer operators where they can go wrong: masked places beside
infinities and NaN, aligned and permuted sources, many groups, offsets out of
range, threads and graphs.  Tolerances as in test_gpu_experts."""
from __future__ import annotations

import ctypes
import math
import threading

import pytest

torch = pytest.importorskip("torch")

import cluster_distributed_shared_gb300 as dh  # noqa: E402
from cluster_distributed_shared_gb300 import experts  # noqa: E402
from test_gpu_experts import (  # noqa: E402,F401
    FLOOR, UNIT, close, cuda_ready, generator, group_exact, route_exact, spans)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- route

@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("experts", [40, 256])
def test_masked_logits_have_no_gradient_beside_infinite_ones(experts, bad, renormalize):
    """An infinite or NaN gradient of a weight stays out of masked logits and
    of other tokens; a missing choice's is not read."""
    g = generator(experts)
    logits = torch.randn(5, experts, generator=g)
    logits[:, ::3] = -math.inf
    logits[3, 7] = math.nan
    logits[4] = -math.inf
    logits[4, 5] = 1.0                              # one choice, the others missing
    dw = torch.randn(5, 4, generator=g)
    dw[1, 2] = bad
    dw[4, 1:] = bad
    ids, w = dh.dsmem_route(logits.cuda(), 4, renormalize=renormalize)
    got = dh.dsmem_route_backward(logits.cuda(), ids, w, dw.cuda(), renormalize=renormalize).cpu()
    masked = ~(logits > -math.inf)
    assert (got[masked] == 0).all()
    assert torch.isfinite(got[[0, 2, 3, 4]]).all() and not torch.isfinite(got[1]).all()


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("pad", [0, 8])
@pytest.mark.parametrize("tokens,experts,k", [(6, 8, 2), (300, 64, 8), (61, 120, 4), (515, 128, 8),
                                              (1026, 256, 8), (7, 248, 32), (66, 384, 6), (35, 512, 10),
                                              (40, 1024, 8)])
def test_route_of_aligned_rows(tokens, experts, k, dtype, pad, renormalize):
    """Rows that are read and written 16 bytes at a time where a lane holds as
    much: whole rows side by side, and rows some aligned distance apart."""
    g = generator(tokens + experts)
    logits = (torch.randn(tokens, experts, generator=g) * 3).to(dtype)
    logits[:, torch.rand(experts, generator=g) < 0.1] = -math.inf
    logits[0, experts // 2] = math.nan
    logits[1] = -math.inf
    logits[2] = 0.25                   # all equal: the lowest indexes
    logits[3, experts - 1] = math.inf
    buf = torch.full((tokens, experts + pad), math.nan, dtype=dtype)
    buf[:, :experts] = logits
    dev = buf.cuda()[:, :experts]
    assert dev.data_ptr() % 16 == 0 and dev.stride(0) * dev.element_size() % 16 == 0
    ids, w = dh.dsmem_route(dev, k, renormalize=renormalize)
    want_ids, want_w, p = route_exact(logits, k, renormalize)
    assert torch.equal(ids.cpu(), want_ids)
    # as test_route_and_gradient's bound, with the argument's rounding: |x - top|
    # is below 32 here, so 16 units of 2^-24 of a weight of 1 at most
    assert (w.cpu().double() - want_w).abs().max() <= (64 + 16) * 2.0 ** -24
    dw = torch.randn(tokens, k, generator=g)
    got = dh.dsmem_route_backward(dev, ids, w, dw.cuda(), renormalize=renormalize)
    d = dw.double()
    dot = torch.where(want_ids >= 0, want_w * d, 0.0).sum(1, keepdim=True)
    full = torch.zeros(tokens, experts, dtype=torch.float64)
    part = want_w * (d - dot) if renormalize else want_w * d
    full.scatter_add_(1, want_ids.clamp(min=0).long(), torch.where(want_ids >= 0, part, 0.0))
    if not renormalize:
        full -= p * dot
    # weights that are off by 80 units, times up to k gradients, and their sums
    bound = UNIT[dtype] * full.abs() + (k + 2) * 96 * 2.0 ** -24 * (d.abs().max() + 1) + FLOOR[dtype]
    assert ((got.cpu().double() - full).abs() <= bound).all()


# ------------------------------------------------------------------- group

@pytest.mark.parametrize("n", [12288, 12289, 262145])
@pytest.mark.parametrize("groups", [17056, 17057, 32768])
@pytest.mark.parametrize("kind", ["uniform", "one", "dropped"])
def test_group_into_very_many(n, groups, kind):
    """Both sides of the counters' shared row and of the sizes that use all SMs."""
    keys = torch.randint(0, groups, (n,), generator=generator(n + groups), dtype=torch.int32)
    if kind == "one":
        keys[:] = groups - 1
    if kind == "dropped":
        keys[::3] = -1
        keys[1::7] = 2 ** 31 - 1
    got = dh.dsmem_group(keys.cuda(), groups)
    for a, b in zip(got, group_exact(keys, groups)):
        assert torch.equal(a.cpu(), b)


# ---------------------------------------------------------------- products

def ragged(g, groups, n, empty, behind):
    """Offsets of n places in `groups` groups, a share of them empty, the last
    `behind` places of none."""
    share = torch.rand(groups, generator=g).double()
    share[torch.rand(groups, generator=g) < empty] = 0
    if not share.any():
        share[groups // 2] = 1
    ends = ((share.cumsum(0) / share.sum()) * (n - behind)).round().int()
    return torch.cat([torch.zeros(1, dtype=torch.int32), ends])


def plain_products(x, w, dy, offsets, row):
    """The three products in 64 bits, each with the sums of magnitudes."""
    n, outer, inner = dy.shape[0], dy.shape[1], x.shape[1]
    y, my = torch.zeros(2, n, outer, dtype=torch.float64)
    dx, mdx = torch.zeros(2, n, inner, dtype=torch.float64)
    dw, mdw = torch.zeros(2, *w.shape, dtype=torch.float64)
    for e, a, b in spans(offsets):
        xr, we, d = x[row[a:b]].double(), w[e].double(), dy[a:b].double()
        y[a:b], my[a:b] = xr @ we.T, xr.abs() @ we.abs().T
        dx[a:b], mdx[a:b] = d @ we, d.abs() @ we.abs()
        dw[e], mdw[e] = d.T @ xr, d.abs().T @ xr.abs()
    return (y, my), (dx, mdx), (dw, mdw)


# Groups: either side of one round of the tables (480) and of the sizes up to
# which the weight gradient's groups are sorted (512), beyond the split over 8
# CTAs (1024), and the most there are, where the tables fill shared memory.
@pytest.mark.parametrize("groups,n,inner,outer,empty", [
    (480, 700, 64, 72, 0.0), (481, 700, 64, 72, 0.0), (481, 300, 64, 72, 0.9), (512, 2000, 72, 64, 0.3),
    (513, 2000, 72, 64, 0.3), (961, 40, 136, 40, 0.0), (1024, 3, 2048, 8, 0.0), (1025, 3, 1024, 8, 0.0),
    (1025, 5000, 40, 136, 0.5), (2048, 2, 1024, 8, 0.0), (2048, 1, 264, 72, 0.0), (2048, 60, 520, 24, 0.9),
    (2048, 9000, 72, 136, 0.2), (2048, 140000, 64, 64, 0.9)])
def test_products_of_many_groups(groups, n, inner, outer, empty):
    g = generator(groups + n)
    behind = n // 10
    offsets = ragged(g, groups, n, empty, behind)
    x = torch.randn(n, inner, generator=g).to(torch.bfloat16)
    w = (torch.randn(groups, outer, inner, generator=g) / math.sqrt(inner)).to(torch.bfloat16)
    dy = torch.randn(n, outer, generator=g).to(torch.bfloat16)
    x[n - behind:], dy[n - behind:] = math.nan, math.nan     # of no group: not read
    order = torch.randperm(n - behind, generator=g).int()
    order = torch.cat([order, torch.full((behind,), -1, dtype=torch.int32)])
    plain = torch.arange(n)
    off, xd, wd, dyd = offsets.cuda(), x.cuda(), w.cuda(), dy.cuda()
    for named in (None, order):
        (y, my), (dx, mdx), (dw, mdw) = plain_products(x, w, dy, offsets, plain if named is None else
                                                       named.clamp(min=0).long())
        rows = {} if named is None else dict(order=named.cuda())
        for out_dtype in (torch.bfloat16, torch.float32):
            close(dh.dsmem_grouped_matmul(xd, wd, off, out_dtype=out_dtype, **rows), y, my, inner)
            if named is None:
                got = dh.dsmem_grouped_matmul(dyd, wd, off, transpose=True, out_dtype=out_dtype)
                close(got, dx, mdx, outer)
            close(dh.dsmem_grouped_matmul_wgrad(dyd, xd, off, out_dtype=out_dtype, **rows), dw, mdw, n)
        del y, my, dx, mdx, dw, mdw


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,groups,fan,inner,outer", [(1, 4, 2, 136, 72), (3, 2, 1, 264, 4096),
                                                           (40, 3, 2, 1003, 517), (300, 7, 3, 129, 65),
                                                           (1300, 16, 1, 800, 520), (3000, 4, 1, 1304, 776)])
def test_input_gradients_of_gathered_rows(tokens, groups, fan, inner, outer, dtype):
    """`transpose` with an `order`: rows of dy by token, each for `fan` places."""
    g = generator(tokens + outer)
    ids = torch.randint(-1 if tokens > 8 else 0, groups, (tokens * fan,), generator=g, dtype=torch.int32)
    offsets, order, _ = group_exact(ids, groups)
    dy = torch.randn(tokens, outer, generator=g).to(dtype)
    w = (torch.randn(groups, outer, inner, generator=g) / math.sqrt(inner)).to(dtype)
    row = torch.where(order < 0, 0, order // fan).long()
    want, size = torch.zeros(2, tokens * fan, inner, dtype=torch.float64)
    for e, a, b in spans(offsets):
        d, we = dy[row[a:b]].double(), w[e].double()
        want[a:b], size[a:b] = d @ we, d.abs() @ we.abs()
    for out_dtype in (dtype, torch.float32):
        got = dh.dsmem_grouped_matmul(dy.cuda(), w.cuda(), offsets.cuda(), order=order.cuda(), fan=fan,
                                      transpose=True, out_dtype=out_dtype)
        close(got, want, size, outer)


@pytest.mark.parametrize("inner", [64, 129])
def test_products_with_permuted_weights(inner):
    """Group strides that are smaller than the row stride, or no multiple of it."""
    g = generator(inner)
    groups, outer, n = 5, 136, 150
    offsets = ragged(g, groups, n, 0.0, 7).cuda()
    w = torch.randn(groups, outer, inner, generator=g).to(torch.bfloat16).cuda()
    x = torch.randn(n, inner, generator=g).to(torch.bfloat16).cuda()
    dy = torch.randn(n, outer, generator=g).to(torch.bfloat16).cuda()
    want = (dh.dsmem_grouped_matmul(x, w, offsets), dh.dsmem_grouped_matmul(dy, w, offsets, transpose=True))
    by_row = torch.empty(outer, groups, inner, dtype=w.dtype, device="cuda").permute(1, 0, 2)
    by_row.copy_(w)
    flat = torch.full((groups * (outer * inner + 24),), math.nan, dtype=w.dtype, device="cuda")
    apart = flat.as_strided((groups, outer, inner), (outer * inner + 24, inner, 1))
    apart.copy_(w)
    lapping = torch.empty(groups - 1 + outer, inner, dtype=w.dtype, device="cuda").normal_()
    lapping = lapping.as_strided((groups, outer, inner), (inner, inner, 1))    # matrices that share rows
    assert by_row.stride(0) < by_row.stride(1) and apart.stride(0) % apart.stride(1) != 0
    for view in (by_row, apart):
        assert torch.equal(dh.dsmem_grouped_matmul(x, view, offsets), want[0])
        assert torch.equal(dh.dsmem_grouped_matmul(dy, view, offsets, transpose=True), want[1])
    whole = lapping.contiguous()
    assert torch.equal(dh.dsmem_grouped_matmul(x, lapping, offsets), dh.dsmem_grouped_matmul(x, whole, offsets))
    assert torch.equal(dh.dsmem_grouped_matmul(dy, lapping, offsets, transpose=True),
                       dh.dsmem_grouped_matmul(dy, whole, offsets, transpose=True))


def guarded(shape, dtype):
    """An output between two margins, and a check that they are untouched."""
    count, margin = math.prod(shape), 4096
    buf = torch.full((count + 2 * margin,), 7.0, dtype=dtype, device="cuda")

    def untouched():
        return bool((buf[:margin] == 7).all() and (buf[margin + count:] == 7).all())

    return buf[margin:margin + count].view(shape), untouched


def entry(name, *args):
    fn = getattr(dh.lib(), name)
    fn.argtypes, fn.restype = experts.SIGNATURES[name], ctypes.c_int
    stream = torch.cuda.current_stream().cuda_stream
    return fn(*[a.data_ptr() if isinstance(a, torch.Tensor) else a for a in args], stream)


@pytest.mark.parametrize("out", [torch.float16, torch.float32])
@pytest.mark.parametrize("inner,outer", [(64, 128), (72, 136), (33, 65)])
@pytest.mark.parametrize("off", [[0, -5, 2 ** 31 - 1, 7], [3, 30, 10, 20], [-1, -1, -1, -1], [0, 0, 0, 2 ** 31 - 1],
                                 [-2 ** 31, 40, 40, 41], [17, 16, 15, 14]])
def test_products_with_offsets_out_of_range(off, inner, outer, out):
    """Ends are clamped to the rows there are and never fall; the first offset
    counts as 0.  Every element is written, and nothing beside them."""
    n, groups = 40, 3
    g = generator(sum(off) + inner)
    ends, last = [0], 0
    for e in off[1:]:
        last = max(last, min(max(e, 0), n))
        ends.append(last)
    x = torch.randn(n, inner, generator=g).to(torch.float16)
    w = torch.randn(groups, outer, inner, generator=g).to(torch.float16)
    dy = torch.randn(n, outer, generator=g).to(torch.float16)
    (y, my), (dx, mdx), (dw, mdw) = plain_products(x, w, dy, torch.tensor(ends), torch.arange(n))
    t = torch.tensor(off, dtype=torch.int32, device="cuda")
    xd, wd, dyd = x.cuda(), w.cuda(), dy.cuda()
    code = experts.F32 if out == torch.float32 else experts.F16
    got, untouched = guarded((n, outer), out)
    assert entry("dsmem_grouped_matmul", xd, n, inner, wd, inner, outer * inner, t, groups, None, 1, n, outer,
                 inner, 0, experts.F16, got, code) == 0
    close(got, y, my, inner)
    assert untouched()
    got, untouched = guarded((n, inner), out)
    assert entry("dsmem_grouped_matmul", dyd, n, outer, wd, inner, outer * inner, t, groups, None, 1, n, outer,
                 inner, 1, experts.F16, got, code) == 0
    close(got, dx, mdx, outer)
    assert untouched()
    got, untouched = guarded((groups, outer, inner), out)
    assert entry("dsmem_grouped_matmul_wgrad", dyd, outer, xd, n, inner, t, groups, None, 1, n, outer, inner,
                 experts.F16, got, code) == 0
    close(got, dw, mdw, n)
    assert untouched()


# ----------------------------------------------------------------- combine

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("width", [8, 129, 264, 2056])
@pytest.mark.parametrize("pad,shift", [(8, 0), (16, 8), (5, 1)])
def test_combine_gradients_of_strided_rows(width, dtype, pad, shift):
    """dy and z as columns of wider tensors, aligned and not."""
    g = generator(width + pad)
    tokens, k = 33, 3
    ids = torch.randint(-1, 5, (tokens, k), generator=g, dtype=torch.int32)
    _, order, position = group_exact(ids.flatten(), 5)
    position = position.view(tokens, k)

    def view(rows):
        buf = torch.full((rows, width + pad), math.nan, dtype=dtype, device="cuda")
        buf[:, shift:shift + width] = torch.randn(rows, width, generator=g).to(dtype).cuda()
        return buf[:, shift:shift + width]

    dy, z, w = view(tokens), view(tokens * k), torch.rand(tokens, k, generator=g).cuda()
    rest = (position.cuda(), order.cuda(), w)
    dz, dw = dh.dsmem_combine_backward(dy, z, *rest)
    ok = position >= 0
    want = torch.zeros(tokens * k, width, dtype=torch.float64)
    want[position[ok].long()] = (w.cpu().double()[..., None] * dy.cpu().double()[:, None, :])[ok]
    close(dz, want, want.abs(), 1)
    rows = torch.where(ok[..., None], z.cpu().double()[position.clamp(min=0).long()], 0.0)
    prod = rows * dy.cpu().double()[:, None, :]
    close(dw, prod.sum(-1), prod.abs().sum(-1), width)


# ------------------------------------------------------- threads and graphs

def layer_step(x, up, logits, k):
    """All the operators, as a training step has them."""
    ids, w = dh.dsmem_route(logits, k)
    off, order, pos = dh.dsmem_group(ids, up.shape[0])
    pos = pos.view(ids.shape)
    h = dh.dsmem_grouped_matmul(x, up, off, order=order, fan=k)
    y = dh.dsmem_combine(h, pos, w)
    dz, dw = dh.dsmem_combine_backward(y, h, pos, order, w)
    dx = dh.dsmem_combine(dh.dsmem_grouped_matmul(dz, up, off, transpose=True), pos)
    dup = dh.dsmem_grouped_matmul_wgrad(dz, x, off, order=order, fan=k)
    dl = dh.dsmem_route_backward(logits, ids, w, dw)
    clipped = [torch.empty_like(dup), torch.empty_like(dl)]
    norm = dh.dsmem_grad_clip([dup, dl], 1.0, out=clipped)
    return [ids, w, off, order, pos, h, y, dz, dw, dx, dup, dl, norm, *clipped]


def layer_inputs(seed, tokens=200, experts=24, inner=72, outer=136):
    g = generator(seed)
    return (torch.randn(tokens, inner, generator=g).to(torch.bfloat16).cuda(),
            torch.randn(experts, outer, inner, generator=g).to(torch.bfloat16).cuda(),
            torch.randn(tokens, experts, generator=g).cuda(), 3)


def test_threads_on_their_own_streams():
    """Calls of many shapes from several threads at once give what one gives."""
    shapes = [dict(tokens=t, experts=e, inner=i, outer=o)
              for t, e, i, o in [(1, 4, 64, 128), (200, 24, 72, 136), (900, 3, 129, 520), (60, 700, 64, 64),
                                 (2500, 5, 264, 304)]]
    inputs = [layer_inputs(7 + j, **s) for j, s in enumerate(shapes)]
    want = [layer_step(*a) for a in inputs]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(4)

    def work(t):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                start.wait()
                for r in range(10):
                    j = (t + r) % len(inputs)
                    got = layer_step(*inputs[j])
                    stream.synchronize()
                    for i, (a, b) in enumerate(zip(got, want[j])):
                        if not torch.equal(a, b):
                            wrong.append((t, r, i))
        except Exception as e:  # noqa: BLE001
            wrong.append((t, repr(e)))

    threads = [threading.Thread(target=work, args=(t,)) for t in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not any(t.is_alive() for t in threads) and not wrong, wrong[:3]


@pytest.mark.parametrize("shape", [dict(tokens=1, experts=4, inner=2048, outer=256), dict(),
                                   dict(tokens=300, experts=7, inner=129, outer=65)])
def test_a_step_in_a_graph(shape):
    """A captured step, replayed on new contents of its inputs (the odd sizes
    take scratch from the pool inside the graph)."""
    x, up, logits, k = layer_inputs(1, **shape)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer_step(x, up, logits, k)               # sets the device up before the capture
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer_step(x, up, logits, k)
    for seed in (2, 3):
        new = layer_inputs(seed, **shape)
        for a, b in zip((x, up, logits), new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(out, layer_step(*new))):
            assert torch.equal(a, b), i


# ---------------------------------------------------------------- refusals

def test_repeated_rows_are_refused():
    """Views that repeat rows or matrices by a stride of 0, and what a norm
    alone is asked for with."""
    h = torch.ones(1, 16, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(2, 8, 16, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    i = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    ones = torch.ones(2, 2, device="cuda")
    z = torch.ones(4, 16, dtype=torch.bfloat16, device="cuda")
    for call in [lambda: dh.dsmem_route(h.expand(4, 16), 2),
                 lambda: dh.dsmem_grouped_matmul(h.expand(4, 16), w, off),
                 lambda: dh.dsmem_grouped_matmul(z, w[:1].expand(2, 8, 16), off),
                 lambda: dh.dsmem_grouped_matmul(z, w[:, :1].expand(2, 8, 16), off),
                 lambda: dh.dsmem_grouped_matmul_wgrad(h.expand(4, 16), z, off),
                 lambda: dh.dsmem_combine(h.expand(4, 16), i),
                 lambda: dh.dsmem_combine_backward(h.expand(2, 16), z, i, i.view(-1), ones),
                 lambda: dh.dsmem_grad_clip([ones], math.inf)]:
        with pytest.raises(dh.DsmemHistError) as e:
            call()
        assert e.value.code == dh.DSMEM_HIST_EINVAL
    most = torch.finfo(torch.float32).max
    assert float(dh.dsmem_grad_clip([ones], most)) == 2.0 and (ones == 1).all()
