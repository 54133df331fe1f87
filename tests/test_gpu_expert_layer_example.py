"""The example's layer answering tokens: a few in one call, and in 4 bits."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from test_gpu_expert_layer import example, plain_layer  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def test_a_few_tokens_in_one_call(example):  # noqa: F811
    layer = example.ExpertLayer(72, 136, 6, 3, seed=5)
    x = torch.randn(40, 72, device="cuda").to(torch.bfloat16)
    y, saved = layer.forward(x)
    want = plain_layer(layer, x, saved[2])[0].detach()
    # the answers' rounding alone: half a unit of 8 bits at most
    assert (layer.decode(x).double().cpu() - want).norm() <= 2.0 ** -8 * want.norm()
    assert torch.equal(layer.decode(x[7]), layer.decode(x[7:8])[0])


def test_in_4_bits(example):  # noqa: F811
    import cluster_distributed_shared_gb300 as dh
    layer = example.ExpertLayer(256, 128, 8, 2, seed=6)
    four = example.FourBitLayer(layer)
    x = torch.randn(33, 256, device="cuda").to(torch.bfloat16)
    # the same layer with what the 4-bit matrices stand for, which bf16 holds exactly
    layer.up = dh.dsmem_mx4_dequantize(*four.up, 256, dtype=torch.bfloat16)
    layer.down = dh.dsmem_mx4_dequantize(*four.down, 128, dtype=torch.bfloat16)
    y, saved = layer.forward(x)
    want = plain_layer(layer, x, saved[2])[0].detach()
    assert (four.decode(x).double().cpu() - want).norm() <= 2.0 ** -8 * want.norm()
    # x's and h's roundings to 4 bits: each under an eighth in the mean square
    assert (four.forward(x).double().cpu() - want).norm() <= 0.25 * want.norm()


def test_the_example_says_how_far_4_bits_are(example, capsys):  # noqa: F811
    example.main(tokens=256, width=128, hidden=64, experts=8, top_k=2, steps=1)
    line = [s for s in capsys.readouterr().out.splitlines() if s.startswith("4-bit")][0]
    few, many = (float(line.split(s)[1].split(",")[0]) for s in ("off by ", "rows by "))
    assert 0 < few < many < 1
