"""An expert layer on the library's operators: one training step, and decoding.

The layer sends every token to the `top_k` best of its experts, each a
two-matrix network, and sums their answers with the router's weights:

    y[t] = sum over j of weights[t, j] * down[e] relu(up[e] x[t]),  e = ids[t, j]

    python examples/expert_layer.py

trains it for a few steps on synthetic tokens, then answers single tokens, and
the same with its matrices in 4 bits.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import cluster_distributed_shared_gb300 as dh  # noqa: E402


class ExpertLayer:
    def __init__(self, width: int, hidden: int, experts: int, top_k: int, dtype=torch.bfloat16,
                 device="cuda", seed: int = 0):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def matrix(*shape):
            t = torch.randn(*shape, generator=g, device=device) / math.sqrt(shape[-1])
            return t.to(dtype)

        self.experts, self.top_k = experts, top_k
        self.router = matrix(experts, width).float()
        self.up = matrix(experts, hidden, width)
        self.down = matrix(experts, width, hidden)

    def forward(self, x):
        """The layer's answers for tokens x [tokens, width], and what the
        backward pass needs of the way there."""
        logits = x.float() @ self.router.t()
        ids, weights = dh.dsmem_route(logits, self.top_k)
        offsets, order, position = dh.dsmem_group(ids, self.experts)
        position = position.view_as(ids)
        hidden = dh.dsmem_grouped_matmul(x, self.up, offsets, order=order, fan=self.top_k)
        active = torch.relu(hidden)
        answers = dh.dsmem_grouped_matmul(active, self.down, offsets)
        y = dh.dsmem_combine(answers, position, weights)
        return y, (x, logits, ids, weights, offsets, order, position, active, answers)

    def backward(self, dy, saved):
        """Gradients (x, router, up, down) for the answers' gradient dy."""
        x, logits, ids, weights, offsets, order, position, active, answers = saved
        d_answers, d_weights = dh.dsmem_combine_backward(dy, answers, position, order, weights)
        d_down = dh.dsmem_grouped_matmul_wgrad(d_answers, active, offsets)
        d_hidden = dh.dsmem_grouped_matmul(d_answers, self.down, offsets, transpose=True)
        d_hidden = d_hidden * (active > 0)
        d_up = dh.dsmem_grouped_matmul_wgrad(d_hidden, x, offsets, order=order, fan=self.top_k)
        d_rows = dh.dsmem_grouped_matmul(d_hidden, self.up, offsets, transpose=True)
        d_logits = dh.dsmem_route_backward(logits, ids, weights, d_weights)
        d_x = dh.dsmem_combine(d_rows, position) + (d_logits @ self.router).to(x.dtype)
        return d_x, d_logits.t() @ x.float(), d_up, d_down

    def train_step(self, x, target, rate: float, max_norm: float = 1.0):
        """One step of gradient descent on the mean squared error; returns the
        loss and the gradients' norm before clipping, on the device."""
        y, saved = self.forward(x)
        error = y.float() - target.float()
        loss = (error * error).mean()
        dy = (error * (2.0 / error.numel())).to(x.dtype)
        _, *grads = self.backward(dy, saved)
        norm = dh.dsmem_grad_clip(grads, max_norm)
        for weight, grad in zip((self.router, self.up, self.down), grads):
            weight.sub_(grad, alpha=rate)
        return loss, norm

    def decode(self, tokens):
        """The answers for a few tokens [up to 64, width], or one [width]."""
        x = tokens.view(-1, tokens.shape[-1])
        y = dh.dsmem_expert_layer(x, x.float() @ self.router.t(), self.up, self.down, self.top_k)
        return y.view_as(tokens)


class FourBitLayer:
    """A trained layer for answering only, with its matrices as microscaled 4-bit
    elements: a quarter of the memory, and of the reading when decoding."""

    def __init__(self, layer: ExpertLayer):
        self.experts, self.top_k, self.router = layer.experts, layer.top_k, layer.router
        self.up, self.down = dh.dsmem_mx4_quantize(layer.up), dh.dsmem_mx4_quantize(layer.down)

    def forward(self, x):
        """Many tokens x [tokens, width], whose rows are multiplied in 4 bits too."""
        ids, weights = dh.dsmem_route(x.float() @ self.router.t(), self.top_k)
        offsets, order, position = dh.dsmem_group(ids, self.experts)
        hidden = dh.dsmem_mx4_grouped_matmul(dh.dsmem_mx4_quantize(x), self.up, offsets, order=order,
                                             fan=self.top_k, out_dtype=x.dtype)
        active = dh.dsmem_mx4_quantize(torch.relu(hidden))
        answers = dh.dsmem_mx4_grouped_matmul(active, self.down, offsets, out_dtype=x.dtype)
        return dh.dsmem_combine(answers, position.view_as(ids), weights)

    decode = ExpertLayer.decode


def main(tokens=4096, width=1024, hidden=512, experts=32, top_k=4, steps=20):
    layer = ExpertLayer(width, hidden, experts, top_k)
    teacher = ExpertLayer(width, hidden, experts, top_k, seed=1)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    for step in range(steps):
        x = torch.randn(tokens, width, generator=g, device="cuda").to(torch.bfloat16)
        loss, norm = layer.train_step(x, teacher.forward(x)[0], rate=2.0)
        if step % 5 == 0 or step == steps - 1:
            print(f"step {step:3d}  loss {float(loss):.5f}  gradient norm {float(norm):.4f}")
    four = FourBitLayer(layer)
    whole, few, many = (t.float() for t in (layer.forward(x)[0][:32], four.decode(x[:32]), four.forward(x)[:32]))
    print(f"4-bit matrices: answers off by {float((few - whole).norm() / whole.norm()):.3f}, with 4-bit rows by "
          f"{float((many - whole).norm() / whole.norm()):.3f}")
    answers = [layer.decode(x[i]) for i in range(4)]
    batch = layer.forward(x[:4])[0]
    print("largest difference of 4 decoded tokens from their batch:",
          float((torch.stack(answers).float() - batch.float()).abs().max()))


if __name__ == "__main__":
    main()
