"""4-bit products of as many groups as leave the tiles' stages just room, or just
none, in shared memory, at each width of tile."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import cluster_distributed_shared_gb300 as dh  # noqa: E402
from test_gpu_mx4_product import check, four_bit, generator  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()


# Tiles 32, 128 and 256 channels wide.  The tables of 2048 groups take 16 KB and a stage
# 22 KB or more, so that each width has at most one such edge.
@pytest.mark.parametrize("n,outer", [(100, 24), (70, 128), (1400, 300)])
@pytest.mark.parametrize("groups", [690, 694, 695, 696, 710, 725, 726, 727, 730, 1024, 2047])
def test_groups_around_the_last_stage_that_fits(groups, n, outer):
    g = generator(groups)
    x, x64 = four_bit(g, n, 300)
    w, w64 = four_bit(g, groups, outer, 300)
    offsets = torch.sort(torch.randint(0, n + 1, (groups + 1,), generator=g)).values.to(torch.int32)
    offsets[0] = 0
    offsets[-1] = n
    got = dh.dsmem_mx4_grouped_matmul(x, w, offsets.cuda(), out_dtype=torch.float32)
    check(got, x64, w64, offsets, torch.arange(n))
