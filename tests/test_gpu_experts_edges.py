"""The expert-layer operators where they can go wrong: masked places beside
infinities and NaN, aligned and permuted sources, many groups, offsets out of
range, threads and graphs.  Tolerances as in test_gpu_experts."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import cluster_distributed_shared_gb300 as dh  # noqa: E402
from test_gpu_experts import (  # noqa: E402,F401
    FLOOR, UNIT, cuda_ready, generator, group_exact, route_exact)

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
