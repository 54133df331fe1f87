"""The whole expert layer for a few tokens, against 64-bit forms.

Tolerances follow from the arithmetic: a value rounded once to a type with unit
roundoff u is off by at most u of itself; a sum of m terms in 32 bits loses at
most one unit in the last place (2^-23) of the sum of magnitudes per addition;
h is held in two 16-bit numbers, together within 2^-16 of it (bf16; f16 2^-22,
and 2^-25 below its normal range)."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import cluster_distributed_shared_gb300 as dh  # noqa: E402
from test_gpu_mx4 import stood_for  # noqa: E402

pytestmark = pytest.mark.gpu

UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
FLOOR = {torch.bfloat16: 2.0 ** -130, torch.float16: 2.0 ** -24}


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


class Layer:
    """Matrices on the device, 16-bit or 4-bit, and their values in 64 bits."""

    def __init__(self, experts, width, hidden, dtype, mx4, gated, seed):
        g = generator(seed)
        self.dtype, self.experts, self.width, self.hidden = dtype, experts, width, hidden

        def make(rows, columns):
            w = torch.randn(experts, rows, columns, generator=g) / math.sqrt(columns)
            if mx4:
                pair = dh.dsmem_mx4_quantize(w.cuda())
                return pair, stood_for(*pair, columns)
            w = w.to(dtype)
            return w.cuda(), w.double()

        self.up, self.up64 = make(hidden, width)
        self.gate, self.gate64 = make(hidden, width) if gated else (None, None)
        self.down, self.down64 = make(width, hidden)

    def run(self, x, logits, top_k, **options):
        return dh.dsmem_expert_layer(x, logits, self.up, self.down, top_k, gate=self.gate, **options)

    def exact(self, x, logits, top_k, activation="relu", renormalize=True):
        """The layer's answers and how far 32-bit sums may be off."""
        x, logits = x.cpu().double(), logits.cpu().double()
        tokens = x.shape[0]
        ids, weights = choices(logits, top_k, renormalize)
        y, off = torch.zeros(tokens, self.width, dtype=torch.float64), torch.zeros(tokens, self.width,
                                                                                   dtype=torch.float64)
        step, two = 2.0 ** -23, (2.0 ** -22 if self.dtype == torch.float16 and not isinstance(self.up, tuple)
                                 else 2.0 ** -16)
        least = 2.0 ** -25 if two < 2.0 ** -20 else 0.0
        for t in range(tokens):
            for j in range(top_k):
                e, w = int(ids[t, j]), float(weights[t, j])
                if e < 0:
                    continue
                u, au = self.up64[e] @ x[t], self.up64[e].abs() @ x[t].abs()
                du = self.width * step * au
                if self.gate64 is None:
                    f, df = u, du
                else:
                    f = self.gate64[e] @ x[t]
                    df = self.width * step * (self.gate64[e].abs() @ x[t].abs())
                a = f * torch.sigmoid(f) if activation == "silu" else f.clamp(min=0)
                da = 1.1 * df + 2.0 ** -20 * a.abs()
                h, dh_ = (a, da) if self.gate64 is None else (a * u, da * u.abs() + (a.abs() + da) * du)
                y[t] += w * (self.down64[e] @ h)
                far = self.down64[e].abs()
                off[t] += w * (far @ (dh_ + (two + 2.0 ** -17) * h.abs()))
                off[t] += far.sum(1) * least + self.hidden * top_k * step * w * (far @ h.abs())
        return y, off

    def check(self, got, want):
        y, off = want
        assert got.dtype == self.dtype and got.shape == y.shape
        g = got.cpu().double()
        bound = UNIT[self.dtype] * (y.abs() + off) + off + FLOOR[self.dtype]
        bad = ~((g - y).abs() <= bound)
        assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} differ, first {bad.nonzero()[0].tolist()}"


def choices(logits, k, renormalize):
    x = torch.where(logits.isnan(), -math.inf, logits)
    best = torch.sort(x, dim=1, descending=True, stable=True)
    ok = best.values[:, :k] > -math.inf
    ids = torch.where(ok, best.indices[:, :k], -1)
    p = torch.nan_to_num(torch.softmax(x, 1), nan=0.0)
    w = torch.where(ok, p.gather(1, ids.clamp(min=0)), 0.0)
    if renormalize:
        w = w / torch.where(w.sum(1, keepdim=True) > 0, w.sum(1, keepdim=True), 1.0)
    return ids, w


def tokens_of(tokens, experts, width, dtype, seed):
    g = generator(seed)
    return torch.randn(tokens, width, generator=g).to(dtype).cuda(), torch.randn(tokens, experts, generator=g).cuda()


SHAPES = [  # tokens, experts, top_k, width, hidden
    (1, 1, 1, 1, 1), (1, 64, 4, 256, 128), (1, 8, 8, 2048, 96), (2, 3, 2, 33, 17), (5, 33, 32, 64, 40),
    (8, 16, 3, 136, 72), (9, 7, 3, 100, 51), (13, 7, 3, 1003, 517), (33, 200, 5, 264, 130), (64, 4, 2, 640, 200),
    (64, 1, 1, 129, 260), (3, 1024, 6, 40, 24), (1, 16, 2, 24, 1100), (64, 32, 32, 72, 40),
    (2, 3, 1, 1, 65536), (2, 3, 2, 65536, 1)]


@pytest.mark.parametrize("gated,activation", [(True, "silu"), (False, "relu"), (True, "relu"), (False, "silu")])
@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,experts,top_k,width,hidden", SHAPES)
def test_layer(tokens, experts, top_k, width, hidden, dtype, mx4, gated, activation):
    seed = tokens * 131 + width
    layer = Layer(experts, width, hidden, dtype, mx4, gated, seed)
    x, logits = tokens_of(tokens, experts, width, dtype, seed + 1)
    renormalize = gated
    got = layer.run(x, logits, top_k, activation=activation, renormalize=renormalize)
    layer.check(got, layer.exact(x, logits, top_k, activation, renormalize))
    again = layer.run(x, logits, top_k, activation=activation, renormalize=renormalize)
    assert torch.equal(got, again)
