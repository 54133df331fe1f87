"""The expert-layer operators where they can go wrong: masked places beside
infinities and NaN, aligned and permuted sources, many groups, offsets out of
range, threads and graphs.  Tolerances as in test_gpu_experts."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import cluster_distributed_shared_gb300 as dh  # noqa: E402
from test_gpu_experts import cuda_ready, generator  # noqa: E402,F401

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
