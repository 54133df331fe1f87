"""Microscaled 4-bit rows on the GPU against the format's definition in 64 bits.

Quantisation is exact: every byte is compared.  The way back rounds once."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import cluster_distributed_shared_gb300 as dh  # noqa: E402

pytestmark = pytest.mark.gpu

VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


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


def quantized(x):
    """The bytes of rows x [rows, columns], from the definition: the nearest
    value by distance, of two equally near ones that with the even code."""
    x = x.detach().cpu().double()
    rows, columns = x.shape
    full = torch.zeros(rows, (columns + 127) // 128 * 128, dtype=torch.float64)
    full[:, :columns] = x
    blocks = full.view(rows, -1, 32)
    most = blocks.abs().amax(2)
    bad = ~torch.isfinite(blocks).all(2)
    safe = torch.where(bad | (most == 0), 1.0, most)
    exponent = torch.floor(torch.log2(safe))
    exponent = torch.where(2.0 ** exponent > safe, exponent - 1, exponent)       # log2 rounds
    exponent = torch.where(2.0 ** (exponent + 1) <= safe, exponent + 1, exponent)
    byte = torch.where(most == 0, torch.zeros_like(most), (exponent - 2 + 127).clamp(min=0))
    byte = torch.where(bad, 255.0, byte)
    scaled = torch.where(bad[..., None], 0.0, blocks) / torch.where(bad, 1.0, 2.0 ** (byte - 127))[..., None]
    distance = (scaled.abs()[..., None].clamp(max=6) - VALUES).abs()
    nearest = distance == distance.amin(-1, keepdim=True)
    code = torch.where(nearest, torch.arange(8), 99).amin(-1)          # the lower of two
    tie = (nearest.sum(-1) == 2) & (code % 2 == 1)
    code = torch.where(tie, code + 1, code) + 8 * torch.signbit(scaled).long()
    code = torch.where(bad[..., None], 0, code).view(rows, -1)
    return (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8), byte.to(torch.uint8)


def stood_for(values, scales, columns):
    """64-bit values of 4-bit rows."""
    v, s = values.cpu().long(), scales.cpu().double()
    table = torch.cat([VALUES, -VALUES])
    each = torch.stack([table[v & 15], table[v >> 4]], -1).flatten(-2)
    scale = torch.where(s == 255, math.nan, 2.0 ** (s - 127))
    return (each * scale.repeat_interleave(32, -1))[..., :columns]


def hard_rows(rows, columns, dtype, seed):
    """Rows whose blocks hold ties, zeros, tiny, huge and mixed values."""
    g = generator(seed)
    x = torch.randn(rows, columns, generator=g) * torch.exp(2 * torch.randn(columns, generator=g))
    x = x.to(dtype)
    low = torch.finfo(dtype)
    x[0] = 0.0
    if rows > 1:   # ties between neighbouring values, at the scale that 6 sets
        x[1] = torch.randint(-28, 29, (columns,), generator=g).to(dtype) / 4
    if rows > 2:
        x[2] = low.max
        x[2, ::3] = -low.max
    if rows > 3:
        x[3] = low.tiny / 2          # below the normal range
    if rows > 4:
        x[4] = -0.0
        x[4, ::40] = 2.0 ** -20
    if rows > 5 and dtype != torch.float16:
        x[5] = torch.randn(columns, generator=g).to(dtype) * 2.0 ** -126
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,columns", [(1, 1), (1, 32), (2, 31), (7, 33), (9, 128), (6, 129), (3, 1000),
                                          (8, 2048), (301, 517), (1, 70001)])
def test_quantize_is_the_definition(rows, columns, dtype):
    x = hard_rows(rows, columns, dtype, rows * 7 + columns)
    values, scales = dh.dsmem_mx4_quantize(x.cuda())
    want_values, want_scales = quantized(x)
    assert torch.equal(scales.cpu(), want_scales)
    assert torch.equal(values.cpu(), want_values)
    exact = stood_for(values, scales, columns)
    for out in (torch.float32, torch.bfloat16, torch.float16):
        back = dh.dsmem_mx4_dequantize(values, scales, columns, dtype=out)
        assert back.shape == x.shape and back.dtype == out
        assert torch.equal(back.cpu(), exact.to(out))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_scale(dtype):
    """Powers of two over the whole range, and the largest values of a block."""
    top = torch.arange(-149, 128, dtype=torch.float64)
    rows = []
    for lead in (1.0, 1.75, 1.9921875):
        block = torch.zeros(len(top), 32, dtype=torch.float64)
        block[:, 5] = lead * 2.0 ** top
        block[:, 6] = -0.3 * 2.0 ** top
        rows.append(block)
    x = torch.cat(rows).to(dtype)
    x = torch.where(torch.isfinite(x), x, 0.0)
    values, scales = dh.dsmem_mx4_quantize(x.cuda())
    want_values, want_scales = quantized(x)
    assert torch.equal(scales.cpu(), want_scales) and torch.equal(values.cpu(), want_values)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_blocks_that_are_not_finite(dtype):
    x = hard_rows(6, 300, dtype, 5)
    x[1, 40] = math.inf
    x[2, 299] = -math.inf
    x[3, 0] = math.nan
    values, scales = dh.dsmem_mx4_quantize(x.cuda())
    want_values, want_scales = quantized(x)
    assert torch.equal(scales.cpu(), want_scales) and torch.equal(values.cpu(), want_values)
    back = dh.dsmem_mx4_dequantize(values, scales, 300).cpu()
    assert back[1, 32:64].isnan().all() and back[3, :32].isnan().all() and back[2, 288:].isnan().all()
    assert int(back.isnan().sum()) == 32 + 32 + 12


def test_all_bytes_come_back():
    """All 256 bytes of two elements beside all 256 scales."""
    values = torch.arange(256, dtype=torch.uint8).repeat(256, 1)                       # 512 elements
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)
    exact = stood_for(values, scales, 512)
    for out in (torch.float32, torch.bfloat16, torch.float16):
        got = dh.dsmem_mx4_dequantize(values.cuda(), scales.cuda(), dtype=out).cpu()
        # 64 bits to 32 first: the scales' values and products are exact there, or infinite
        assert torch.equal(got.nan_to_num(7e7), exact.float().to(out).nan_to_num(7e7))


def test_rows_with_strides_and_odd_bases():
    g = generator(3)
    for dtype in (torch.float32, torch.bfloat16):
        wide = torch.randn(40, 333, generator=g).to(dtype)
        for view in (wide[:, :200], wide[:, 3:300], wide[::2, 1:65], wide[5:6, 8:168]):
            dev = wide.cuda()[:, :]
            dev = torch.as_strided(dev, view.shape, view.stride(), view.storage_offset())
            values, scales = dh.dsmem_mx4_quantize(dev)
            want_values, want_scales = quantized(view)
            assert torch.equal(values.cpu(), want_values) and torch.equal(scales.cpu(), want_scales)


def test_leading_dimensions():
    x = torch.randn(3, 5, 2, 130, generator=generator(4))
    values, scales = dh.dsmem_mx4_quantize(x.cuda())
    assert values.shape == (3, 5, 2, 128) and scales.shape == (3, 5, 2, 8)
    want = quantized(x.view(-1, 130))
    assert torch.equal(values.cpu().view(-1, 128), want[0]) and torch.equal(scales.cpu().view(-1, 8), want[1])
    back = dh.dsmem_mx4_dequantize(values, scales, 130, dtype=torch.float16)
    assert back.shape == x.shape
    none = dh.dsmem_mx4_quantize(x[:0].cuda())
    assert none[0].shape == (0, 5, 2, 128) and dh.dsmem_mx4_dequantize(*none, 130).shape == (0, 5, 2, 130)
    one = dh.dsmem_mx4_quantize(x[0, 0, 0].cuda())
    assert torch.equal(one[0], values[0, 0, 0]) and torch.equal(one[1], scales[0, 0, 0])


def test_nothing_around_the_outputs_is_written():
    lib = dh.lib()
    rows, columns = 5, 200
    x = torch.randn(rows, columns, generator=generator(6)).cuda()
    values = torch.full((rows * 128 + 64,), 77, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows * 8 + 64,), 77, dtype=torch.uint8, device="cuda")
    out = torch.full((rows * columns + 64,), 77.0, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    from cluster_distributed_shared_gb300 import experts
    dh.dsmem_mx4_quantize(x)   # declares the entries' types
    assert lib.dsmem_mx4_quantize(x.data_ptr(), experts.F32, rows, columns, columns, values.data_ptr() + 32,
                                  scales.data_ptr() + 32, stream) == 0
    assert lib.dsmem_mx4_dequantize(values.data_ptr() + 32, scales.data_ptr() + 32, rows, columns, experts.F32,
                                    out.data_ptr() + 128, stream) == 0
    want = quantized(x)
    assert torch.equal(values[32:-32].view(rows, 128).cpu(), want[0])
    assert torch.equal(scales[32:-32].view(rows, 8).cpu(), want[1])
    for t in (values, scales, out):
        assert (t[:32] == 77).all() and (t[-32:] == 77).all()


def test_more_than_32_bits_of_elements():
    """Rows past element 2^32 of their tensor."""
    rows, columns = 1100000, 4096
    x = torch.zeros(rows, columns, dtype=torch.bfloat16, device="cuda")
    mark = torch.randn(3, columns, generator=generator(8)).to(torch.bfloat16)
    at = [0, 2 ** 20 + 12345, rows - 1]
    for i, r in enumerate(at):
        x[r] = mark[i].cuda()
    values, scales = dh.dsmem_mx4_quantize(x)
    want = quantized(mark)
    assert torch.equal(values[at].cpu(), want[0]) and torch.equal(scales[at].cpu(), want[1])
    assert int((scales != 0).any(1).sum()) == 3
    x.fill_(1.0)
    back = dh.dsmem_mx4_dequantize(values, scales, columns, dtype=torch.bfloat16)
    assert torch.equal(back[at].cpu().double(), stood_for(*want, columns))
    assert int((back != 0).any(1).sum()) == 3
