"""Layers of f16 matrices whose hidden values lie below f16's normal range, or
beyond its largest number, against 64-bit forms.

A result is off by its own rounding, half a step of f16 (2^-11 of it, 2^-25 where it
is subnormal), by 2^-22 of each hidden value or 2^-39 of the largest one of its token
and expert, and by at most one unit in the last place (2^-23) of the sum of
magnitudes for each 32-bit addition: width of them in a hidden value, two for each
of a channel's hidden * top_k terms."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import cluster_distributed_shared_gb300 as dh  # noqa: E402
from test_gpu_expert_layer_few import choices, generator, tokens_of  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda_ready():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    yield
    torch.cuda.synchronize()


def exact(x, logits, up, gate, down, top_k, activation, renormalize):
    """The layer in 64 bits, and how far its 32-bit sums and h may be off."""
    ids, weights = choices(logits.cpu().double(), top_k, renormalize)
    x, up, gate, down = (t.cpu().double() if t is not None else None for t in (x, up, gate, down))
    width, hidden, step = up.shape[2], up.shape[1], 2.0 ** -23
    y, off = torch.zeros_like(x), torch.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(top_k):
            e, w = int(ids[t, j]), float(weights[t, j])
            if e < 0:
                continue
            u, du = up[e] @ x[t], width * step * (up[e].abs() @ x[t].abs())
            f, df = (u, du) if gate is None else (gate[e] @ x[t], width * step * (gate[e].abs() @ x[t].abs()))
            a = f * torch.sigmoid(f) if activation == "silu" else f.clamp(min=0)
            # silu's slope is at most 1.1; the function itself, the weight and h's product are a few units off
            da = 1.1 * df + 2.0 ** -20 * a.abs()
            h, dh_ = (a, da) if gate is None else (a * u, da * u.abs() + (a.abs() + da) * du)
            far = down[e].abs()
            y[t] += w * (down[e] @ h)
            off[t] += w * (far @ (dh_ + (2.0 ** -22 + 2.0 ** -20) * h.abs() + 2.0 ** -39 * h.abs().max()))
            off[t] += 2 * hidden * top_k * step * w * (far @ h.abs())
    return y, off


def matrices(seed, experts, width, hidden, gated, size):
    g = generator(seed)

    def make(rows, columns, by):
        return (torch.randn(experts, rows, columns, generator=g) * (by / math.sqrt(columns))).half().cuda()

    return make(hidden, width, 1.0), make(hidden, width, 1.0) if gated else None, make(width, hidden, size)


def check(got, y, off):
    bound = (2.0 ** -11 * (y.abs() + off)).clamp(min=2.0 ** -25) + off
    bad = ~((got.cpu().double() - y).abs() <= bound)
    assert got.dtype == torch.float16
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} differ, first {bad.nonzero()[0].tolist()}"


# Sizes of x and of down: answers near one from ever smaller hidden values, last from those beyond 65504.
SIZES = [(0.03, 4.0), (0.01, 64.0), (0.003, 512.0), (2.0 ** -12, 8192.0), (2.0 ** -17, 32768.0), (2.0 ** 13, 2.0 ** -14)]


@pytest.mark.parametrize("gated,activation,renormalize", [(True, "silu", True), (True, "relu", False),
                                                          (False, "silu", False)])
@pytest.mark.parametrize("size,back", SIZES)
@pytest.mark.parametrize("tokens,experts,top_k,width,hidden", [(1, 8, 2, 64, 40), (7, 100, 3, 136, 65), (20, 4, 2, 33, 96),
                                                               (64, 2, 1, 72, 136)])
def test_hidden_values_of_any_size(tokens, experts, top_k, width, hidden, size, back, gated, activation, renormalize):
    up, gate, down = matrices(tokens + width, experts, width, hidden, gated, back)
    x, logits = tokens_of(tokens, experts, width, torch.float16, tokens)
    x = x * size
    got = dh.dsmem_expert_layer(x, logits, up, down, top_k, gate=gate, activation=activation, renormalize=renormalize)
    y, off = exact(x, logits, up, gate, down, top_k, activation, renormalize)
    check(got, y, off)


@pytest.mark.parametrize("size,back", [(0.03, 8.0), (0.01, 64.0), (0.003, 512.0), (2.0 ** -17, 32768.0)])
@pytest.mark.parametrize("gated", [True, False])
def test_a_deep_layer_of_small_tokens(size, back, gated):
    """1024 hidden values a channel, in the mean square: beside the output's own
    rounding sums of m terms of either sign lose about sqrt(m) 2^-24, h 2^-22."""
    up, gate, down = matrices(5, 8, 512, 1024, gated, back)
    x, logits = tokens_of(6, 8, 512, torch.float16, 6)
    x = x * size
    got = dh.dsmem_expert_layer(x, logits, up, down, 4, gate=gate, activation="silu").cpu().double()
    y, _ = exact(x, logits, up, gate, down, 4, "silu", True)
    least = (y.half().double() - y).norm() / y.norm()
    assert (got - y).norm() / y.norm() <= 1.01 * least + math.sqrt(2 * 4 * 1024) * 2.0 ** -24 + 2.0 ** -20


def test_small_routing_weights():
    """A hidden value times a small weight: one expert far ahead of the others, all
    chosen, and only a small one's matrices not zero."""
    up, gate, down = matrices(7, 6, 96, 200, True, 8192.0)
    for m in (up, down):
        m[0] = 0
    x, logits = tokens_of(9, 6, 96, torch.float16, 8)
    logits[:, 0] += 14.0
    got = dh.dsmem_expert_layer(x, logits, up, down, 6, gate=gate, activation="silu")
    y, off = exact(x, logits, up, gate, down, 6, "silu", True)
    check(got, y, off)


def test_infinite_and_undefined_hidden_values_stay_with_their_tokens():
    up, gate, down = matrices(9, 3, 72, 100, False, 1.0)
    down.abs_()
    x, logits = tokens_of(12, 3, 72, torch.float16, 10)
    want = dh.dsmem_expert_layer(x, logits, up, down, 2)
    up.clamp_(min=2.0 ** -6)                      # a row without zeros
    clean = dh.dsmem_expert_layer(x, logits, up, down, 2)
    x[3, 5], x[11, 71] = math.inf, math.nan
    got = dh.dsmem_expert_layer(x, logits, up, down, 2)
    rest = [t for t in range(12) if t not in (3, 11)]
    assert want.isfinite().all() and torch.equal(got[rest], clean[rest])
    whole = (down > 0).all(2)                     # channels of which no element is 0
    ids, _ = dh.dsmem_route(logits, 2)
    channels = whole[ids[3].long()].all(0)
    assert (got[3][channels] == math.inf).all() and got[11].isnan().all()


def small_layers():
    """Layers of small f16 tokens: (x, logits, up, gate, down, top_k) each."""
    sizes = [(1, 8, 2, 136, 65, 0.003), (24, 5, 3, 64, 200, 2.0 ** -12), (64, 16, 2, 72, 40, 1.0)]
    made = []
    for i, (tokens, experts, k, width, hidden, size) in enumerate(sizes):
        up, gate, down = matrices(20 + i, experts, width, hidden, True, 64.0)
        x, logits = tokens_of(tokens, experts, width, torch.float16, 30 + i)
        made.append((x * size, logits, up, gate, down, k))
    return made


def answer(x, logits, up, gate, down, k):
    return dh.dsmem_expert_layer(x, logits, up, down, k, gate=gate, activation="silu")


def test_captured_layers_in_turn_and_together():
    inputs = small_layers()
    for a in inputs:
        check(answer(*a), *exact(*a[:2], a[2], a[3], a[4], a[5], "silu", True))
    graphs, outs = [], []
    for a in inputs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(answer(*a))
        graphs.append(graph)
    for size in (1.0, 2.0 ** -6, 2.0 ** 6):
        for a in inputs:
            a[0].mul_(size)
        streams = [torch.cuda.Stream() for _ in graphs]
        for rounds in range(3):
            torch.cuda.synchronize()
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for a, got in zip(inputs, outs):
            assert torch.equal(got, answer(*a))


def test_calls_of_several_threads():
    import threading
    inputs = small_layers()
    want = [answer(*a) for a in inputs]
    torch.cuda.synchronize()
    wrong, start = [], threading.Barrier(4)

    def work(t):
        try:
            stream = torch.cuda.Stream() if t % 2 else torch.cuda.default_stream()
            with torch.cuda.stream(stream):
                start.wait()
                for r in range(20):
                    j = (t + r) % len(inputs)
                    got = answer(*inputs[j])
                    stream.synchronize()
                    if not torch.equal(got, want[j]):
                        wrong.append((t, r))
        except Exception as e:  # noqa: BLE001
            wrong.append((t, repr(e)))

    threads = [threading.Thread(target=work, args=(t,)) for t in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not any(t.is_alive() for t in threads) and not wrong, wrong[:3]
