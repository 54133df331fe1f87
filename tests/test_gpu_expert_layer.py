"""The expert layer of examples/expert_layer.py: its operators together, against
the same layer in plain torch with automatic differentiation in 64 bits."""
from __future__ import annotations

import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location(
        "expert_layer", os.path.join(ROOT, "examples", "expert_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain_layer(layer, x, ids):
    """The layer in 64 bits, every expert on every token, on the choices `ids`."""
    leaves = [t.double().cpu().requires_grad_() for t in (x, layer.router, layer.up, layer.down)]
    xd, router, up, down = leaves
    chosen = (xd @ router.t()).gather(1, ids.cpu().long())
    weights = torch.softmax(chosen, 1)
    y = torch.zeros_like(xd)
    for j in range(ids.shape[1]):
        e = ids[:, j].cpu().long()
        hidden = torch.relu(torch.einsum("thd,td->th", up[e], xd))
        y = y + weights[:, j:j + 1] * torch.einsum("tdh,th->td", down[e], hidden)
    return y, leaves


@pytest.mark.parametrize("tokens,width,hidden,experts,top_k", [(1, 64, 40, 4, 2), (50, 72, 136, 6, 3)])
def test_layer_and_gradients(example, tokens, width, hidden, experts, top_k):
    layer = example.ExpertLayer(width, hidden, experts, top_k, seed=tokens)
    g = torch.Generator().manual_seed(tokens)
    x = torch.randn(tokens, width, generator=g).to(torch.bfloat16).cuda()
    dy = torch.randn(tokens, width, generator=g).to(torch.bfloat16).cuda()
    y, saved = layer.forward(x)
    want, leaves = plain_layer(layer, x, saved[2])
    want.backward(dy.double().cpu())
    # Up to six roundings to 8 significant bits lie between an input and a
    # gradient, each 2^-9 of the typical value: compared in the mean.
    for got, ref in zip((y, *layer.backward(dy, saved)), (want.detach(), *[t.grad for t in leaves])):
        error = (got.double().cpu() - ref).norm() / ref.norm()
        assert error <= 6 * 2.0 ** -9 * 2, float(error)


def test_training_lowers_the_loss_and_decoding_agrees(example, capsys):
    example.main(tokens=512, width=128, hidden=64, experts=8, top_k=2, steps=11)
    lines = capsys.readouterr().out.splitlines()
    losses = [float(line.split("loss")[1].split()[0]) for line in lines if "loss" in line]
    assert losses[-1] < losses[0]
    # the sums' order may differ with the number of rows: a unit of bfloat16 of values up to 4
    assert float(lines[-1].split(":")[1]) <= 4 * 2.0 ** -8


def test_layer_on_another_stream(example):
    layer = example.ExpertLayer(128, 64, 8, 2)
    x = torch.randn(300, 128, device="cuda").to(torch.bfloat16)
    want = layer.forward(x)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = [layer.forward(x)[0] for _ in range(8)]
    torch.cuda.current_stream().wait_stream(side)
    for t in got:
        assert torch.equal(t, want)
