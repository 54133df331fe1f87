"""4-bit matrices whose scales are not a number, or lie at the ends of their range,
inside the experts that a layer's tokens chose."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import cluster_distributed_shared_gb300 as dh  # noqa: E402
from test_gpu_expert_layer_few import Layer, generator, tokens_of  # noqa: E402
from test_gpu_mx4 import stood_for  # noqa: E402
from test_gpu_mx4_product import check as check_product  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens", [1, 12, 40])
@pytest.mark.parametrize("name,row,block", [("down", 7, 3), ("down", 0, 0), ("down", 199, 9), ("up", 11, 2),
                                            ("up", 299, 6), ("gate", 0, 0), ("gate", 150, 5)])
def test_a_block_that_is_not_a_number(name, row, block, tokens, dtype):
    """In a row of down it is the channel's of the expert's tokens, in up or gate all
    of their channels; every other answer keeps its bits."""
    layer = Layer(3, 200, 300, dtype, True, True, 5)
    x, logits = tokens_of(tokens, 3, 200, dtype, 6)
    logits[0, 1] = 5.0
    clean = layer.run(x, logits, 2)
    ids, _ = dh.dsmem_route(logits, 2)
    chose = (ids == 1).any(1)
    getattr(layer, name)[1][1, row, block] = 255
    got = layer.run(x, logits, 2)
    touched = torch.zeros_like(got, dtype=torch.bool)
    if name == "down":
        touched[chose, row] = True
    else:
        touched[chose] = True
    assert chose[0] and clean.isfinite().all()
    assert torch.equal(got.isnan(), touched) and torch.equal(got[~touched], clean[~touched])


@pytest.mark.parametrize("up,down", [(0, 250), (1, 252), (2, 240), (245, 5), (247, 0), (128, 129), (129, 126)])
@pytest.mark.parametrize("tokens", [2, 12])
def test_layers_of_scales_at_the_ends(tokens, up, down):
    """Blocks of one scale each, up to the largest that quantisation gives (252), that
    make up for one another."""
    layer = Layer(2, 128, 256, torch.bfloat16, True, False, 7)
    for name, byte, columns in (("up", up, 128), ("down", down, 256)):
        pair = getattr(layer, name)
        pair[1].fill_(byte)
        setattr(layer, name + "64", stood_for(*pair, columns))
    x, logits = tokens_of(tokens, 2, 128, torch.bfloat16, 8)
    layer.check(layer.run(x, logits, 1), layer.exact(x, logits, 1))


@pytest.mark.parametrize("rows,matrix", [(0, 250), (1, 252), (252, 0), (252, 2), (250, 4), (127, 127), (100, 154)])
def test_products_of_scales_at_the_ends(rows, matrix):
    g = generator(9)
    x = dh.dsmem_mx4_quantize(torch.randn(40, 256, generator=g).cuda())
    w = dh.dsmem_mx4_quantize((torch.randn(1, 48, 256, generator=g) * math.sqrt(0.5)).cuda())
    x[1].fill_(rows)
    w[1].fill_(matrix)
    offsets = torch.tensor([0, 40], dtype=torch.int32)
    got = dh.dsmem_mx4_grouped_matmul(x, w, offsets.cuda(), out_dtype=torch.float32)
    check_product(got, stood_for(*x, 256), stood_for(*w, 256), offsets, torch.arange(40))
