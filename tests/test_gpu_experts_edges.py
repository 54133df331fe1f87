"""The expert-layer operators where they can go wrong: masked places beside
infinities and NaN, aligned and permuted sources, many groups, offsets out of
range, threads and graphs.  Tolerances as in test_gpu_experts."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import cluster_distributed_shared_gb300 as dh  # noqa: E402
from test_gpu_experts import cuda_ready, generator, group_exact  # noqa: E402,F401

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
