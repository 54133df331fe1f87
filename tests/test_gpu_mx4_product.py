"""Products of 4-bit rows and matrices grouped by key, against 64-bit products of
what they stand for.  A result is off by its own rounding and, for each of its
terms' 32-bit additions, by at most one unit in the last place (2^-23) of the
sum of magnitudes."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import cluster_distributed_shared_gb300 as dh  # noqa: E402
from test_gpu_mx4 import stood_for  # noqa: E402

pytestmark = pytest.mark.gpu

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
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


def four_bit(g, *shape):
    """A pair on the device, and its values in 64 bits."""
    x = torch.randn(*shape, generator=g) * torch.exp(torch.randn(shape[-1], generator=g))
    pair = dh.dsmem_mx4_quantize(x.cuda())
    return pair, stood_for(*pair, shape[-1])


def check(got, x, w, offsets, rows):
    """got[p] against x[rows[p]] w[g]^T; rows below 0 are none."""
    off = offsets.tolist()
    want = torch.zeros(got.shape, dtype=torch.float64)
    size = torch.zeros(got.shape, dtype=torch.float64)
    xs = torch.cat([x, torch.zeros(1, x.shape[1], dtype=torch.float64)])
    for g in range(w.shape[0]):
        a, b = off[g], off[g + 1]
        if b > a:
            src = xs[rows[a:b]]
            want[a:b] = src @ w[g].t()
            size[a:b] = src.abs() @ w[g].abs().t()
    bound = UNIT[got.dtype] * want.abs() + x.shape[1] * 2.0 ** -23 * (1 + UNIT[got.dtype]) * size + FLOOR[got.dtype]
    bad = ~((got.cpu().double() - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} differ, first {bad.nonzero()[0].tolist()}"


CASES = [  # group sizes, rows behind the last group, inner, outer
    ([1], 0, 32, 8), ([1], 0, 1, 1), ([5], 0, 256, 128), ([3, 0, 7], 2, 100, 40), ([128], 0, 128, 256),
    ([127, 129, 1], 3, 300, 130), ([0, 0, 0], 5, 64, 33), ([200, 0, 57, 300], 0, 1003, 517),
    ([64] * 20, 11, 640, 264), ([1, 0, 2, 1] * 16, 0, 2048, 96), ([700], 0, 384, 1100), ([33] * 5, 0, 4096, 48),
    # enough tiles for 256 channels each: several a CTA, ragged ones, many groups without rows
    ([1, 129, 0, 40, 128] * 10, 7, 300, 2050), ([5] * 300, 0, 1100, 520), ([2, 0] * 300 + [1], 3, 96, 300),
    # several row tiles of the same channels, at each width of tile
    ([600, 129, 0, 333] * 6, 0, 1100, 2050), ([700, 300] * 3, 5, 1600, 2050), ([700, 300], 0, 2048, 1100)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("sizes,behind,inner,outer", CASES)
def test_rows_in_place(sizes, behind, inner, outer, dtype):
    g = generator(inner + outer)
    n = sum(sizes) + behind
    x, x64 = four_bit(g, n, inner)
    w, w64 = four_bit(g, len(sizes), outer, inner)
    offsets = torch.tensor([0, *sizes]).cumsum(0).to(torch.int32)
    got = dh.dsmem_mx4_grouped_matmul(x, w, offsets.cuda(), out_dtype=dtype)
    check(got, x64, w64, offsets, torch.arange(n))
    assert torch.equal(got, dh.dsmem_mx4_grouped_matmul(x, w, offsets.cuda(), out_dtype=dtype))


@pytest.mark.parametrize("fan", [1, 3])
@pytest.mark.parametrize("sizes,behind,inner,outer", CASES)
def test_rows_of_an_order(sizes, behind, inner, outer, fan):
    g = generator(inner * 3 + outer + fan)
    n, sources = sum(sizes) + behind, 37
    x, x64 = four_bit(g, sources, inner)
    w, w64 = four_bit(g, len(sizes), outer, inner)
    offsets = torch.tensor([0, *sizes]).cumsum(0).to(torch.int32)
    order = torch.randint(0, sources * fan, (n,), generator=g).to(torch.int32)
    if n > 4:
        order[1], order[2], order[n // 2] = -1, sources * fan, 2 ** 31 - 1     # no rows of x
        order[3] = -2 ** 31
    rows = torch.where(order < 0, -1, order // fan).long()
    rows = torch.where(rows < sources, rows, -1)
    got = dh.dsmem_mx4_grouped_matmul(x, w, offsets.cuda(), order=order.cuda(), fan=fan, out_dtype=torch.float32)
    check(got, x64, w64, offsets, rows)


@pytest.mark.parametrize("offsets", [[5, 3, -7, 100, 9], [0, 50, 20, 60, 40], [0, 0, 0, 0, 0], [-3, 10, 10, 64, 65]])
def test_offsets_are_clamped(offsets):
    """Offsets out of range or order count as the running maximum within [0, n]."""
    g = generator(7)
    x, x64 = four_bit(g, 64, 160)
    w, w64 = four_bit(g, 4, 72, 160)
    ends = [0]
    for o in offsets[1:]:
        ends.append(max(ends[-1], min(max(o, 0), 64)))
    got = dh.dsmem_mx4_grouped_matmul(x, w, torch.tensor(offsets, dtype=torch.int32).cuda(),
                                      out_dtype=torch.float32)
    check(got, x64, w64, torch.tensor(ends), torch.arange(64))


def test_what_is_not_a_number_stays_in_its_rows_and_columns():
    g = generator(9)
    x = torch.randn(150, 300, generator=g)
    w = torch.randn(2, 70, 300, generator=g)
    x[4, 33], x[149, 299] = math.nan, math.inf
    w[1, 69, 0] = -math.inf
    xp, wp = dh.dsmem_mx4_quantize(x.cuda()), dh.dsmem_mx4_quantize(w.cuda())
    offsets = torch.tensor([0, 20, 140], dtype=torch.int32)
    got = dh.dsmem_mx4_grouped_matmul(xp, wp, offsets.cuda(), out_dtype=torch.float32).cpu()
    nan = torch.zeros(150, 70, dtype=torch.bool)
    nan[4] = True
    nan[20:140, 69] = True
    assert torch.equal(got.isnan(), nan)
    assert (got[140:] == 0).all()
    clean = torch.where(nan, 0.0, got)
    x64 = stood_for(*xp, 300).nan_to_num(0.0)
    w64 = stood_for(*wp, 300).nan_to_num(0.0)
    want = torch.cat([x64[:20] @ w64[0].t(), x64[20:140] @ w64[1].t(), torch.zeros(10, 70)])
    assert torch.allclose(clean.double(), torch.where(nan, 0.0, want), rtol=1e-4, atol=1e-4)


def test_wide_range_of_scales():
    """Scales far from 1 on both sides that cancel in the product."""
    g = generator(10)
    x = torch.randn(40, 256, generator=g) * 2.0 ** 60
    w = torch.randn(1, 48, 256, generator=g) * 2.0 ** -70
    xp, wp = dh.dsmem_mx4_quantize(x.cuda()), dh.dsmem_mx4_quantize(w.cuda())
    offsets = torch.tensor([0, 40], dtype=torch.int32)
    got = dh.dsmem_mx4_grouped_matmul(xp, wp, offsets.cuda(), out_dtype=torch.float32)
    check(got, stood_for(*xp, 256), stood_for(*wp, 256), offsets, torch.arange(40))
