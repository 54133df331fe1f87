"""The expert-layer operators at the ends of their ranges: sizes that the C
entries' 32-bit arguments cannot hold, and the widest rows they can."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

import cluster_distributed_shared_gb300 as dh  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def test_sizes_past_32_bits_are_refused():
    """None of them is taken modulo 2^32."""
    past = 2 ** 32
    i = torch.zeros(4, dtype=torch.int32, device="cuda")
    f = torch.zeros(1, 8, device="cuda")
    h = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(2, 8, 16, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")

    def wide(dtype=torch.bfloat16):               # no rows, so no memory
        return torch.empty(0, past + 16, dtype=dtype, device="cuda")

    no = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    real = torch.empty(0, 2, device="cuda")
    for call in [
        lambda: dh.dsmem_route(f, past + 2),
        lambda: dh.dsmem_route(f, 2 - past),
        lambda: dh.dsmem_route(f, -1),
        lambda: dh.dsmem_route(wide(torch.float32), 2),
        lambda: dh.dsmem_route_backward(wide(torch.float32), no, real, real),
        lambda: dh.dsmem_group(i, past + 4),
        lambda: dh.dsmem_group(i, 4 - past),
        lambda: dh.dsmem_grouped_matmul(h, w, off, order=i, fan=past + 1),
        lambda: dh.dsmem_grouped_matmul(h, w, off, order=i, fan=1 - past),
        lambda: dh.dsmem_grouped_matmul_wgrad(h, h, off, order=i, fan=past + 1),
        lambda: dh.dsmem_grouped_matmul_wgrad(wide(), h[:0], off),
        lambda: dh.dsmem_grouped_matmul_wgrad(h[:0], wide(), off),
        lambda: dh.dsmem_combine(wide(), no),
        lambda: dh.dsmem_combine_backward(wide(), wide(), no, i[:0], real),
    ]:
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("width", [65535 * 512 + 515, 65535 * 2048 + 2056])
def test_combine_of_rows_wider_than_one_grid(width):
    """More pieces of a row than a grid's second extent, element by element
    (an odd width) and in 16-byte vectors.  Products by 0.5 and the sums are exact."""
    g = torch.Generator(device="cuda").manual_seed(width)
    z = torch.randn(1, width, generator=g, device="cuda", dtype=torch.bfloat16)
    position = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    half = torch.full((1, 1), 0.5, device="cuda")
    assert torch.equal(dh.dsmem_combine(z, position, half), z * 0.5)
    ones = torch.zeros_like(z)
    ones[:, ::1024] = 1.0
    dz, dw = dh.dsmem_combine_backward(ones, ones, position, position.view(1), half)
    assert torch.equal(dz, ones * 0.5) and float(dw) == float(ones.sum(dtype=torch.float64))


def test_products_of_rows_longer_than_2_to_30():
    """Gathered rows of more than 2^30 elements: all of a row is read, its
    first elements and its last.  The products and sums are exact."""
    long = 2 ** 30 + 72
    x = torch.zeros(1, long, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(1, 1, long, dtype=torch.bfloat16, device="cuda")
    x[0, :64], x[0, -8:] = 1.0, 2.0
    w[0, 0, :64], w[0, 0, -8:] = 0.5, 1.0
    off = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    order = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = dh.dsmem_grouped_matmul(x, w, off, order=order, out_dtype=torch.float32)
    assert y.item() == 64 * 0.5 + 8 * 2.0
    dy = torch.full((1, 1), 2.0, dtype=torch.bfloat16, device="cuda")
    dw = dh.dsmem_grouped_matmul_wgrad(dy, x, off, order=order)
    assert torch.equal(dw.view(-1), x.view(-1) * 2.0)
    dw = dh.dsmem_grouped_matmul_wgrad(x, dy, off, order=order)
    assert torch.equal(dw.view(-1), x.view(-1) * 2.0)
