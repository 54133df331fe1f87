"""The whole expert layer and the 4-bit entries where they can go wrong: logits
that are masked or not finite, experts that nobody chose, strides and bases,
scales at the ends of their range, streams, threads, graphs, and refusals."""
from __future__ import annotations

import math
import threading

import pytest

torch = pytest.importorskip("torch")

import cluster_distributed_shared_gb300 as dh  # noqa: E402
from cluster_distributed_shared_gb300 import experts as entries  # noqa: E402
import test_gpu_expert_layer_few as few  # noqa: E402
from test_gpu_expert_layer_few import Layer, generator, tokens_of  # noqa: E402
from test_gpu_mx4 import stood_for  # noqa: E402
from test_gpu_mx4_product import check as check_product, four_bit  # noqa: E402

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


# ---------------------------------------------------------------- the layer

def check_as_routed(monkeypatch, layer, x, logits, top_k, renormalize, **options):
    """The layer's answer against the formula with dsmem_route's choices."""
    ids, weights = (t.cpu() for t in dh.dsmem_route(logits, top_k, renormalize=renormalize))
    monkeypatch.setattr(few, "choices", lambda *_: (ids, weights))
    got = layer.run(x, logits, top_k, renormalize=renormalize, **options)
    layer.check(got, layer.exact(x, logits, top_k, options.get("activation", "relu"), renormalize))
    return got, ids


@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("experts", [9, 100, 300])
def test_masked_and_tied_logits(monkeypatch, experts, kind, mx4, renormalize):
    """Rows with nothing, with less than top_k, with the type's lowest value, NaN
    and ties, of logits that are a view with a stride."""
    layer = Layer(experts, 72, 40, torch.bfloat16, mx4, True, experts)
    x, _ = tokens_of(14, experts, 72, torch.bfloat16, 3)
    logits = torch.randn(14, experts + 5, generator=generator(4)).to(kind)[:, 2:-3]
    logits[0] = -math.inf
    logits[1] = math.nan
    logits[2, 1:] = -math.inf
    logits[3] = torch.finfo(kind).min
    logits[4] = 1.0
    logits[5, ::2] = -math.inf
    logits[6, 3:] = math.nan
    logits[7, :4] = torch.finfo(kind).max
    logits[8, :] = -math.inf
    logits[8, -1] = torch.finfo(kind).min
    got, ids = check_as_routed(monkeypatch, layer, x, logits.cuda(), 4, renormalize, activation="silu")
    assert (got[:2] == 0).all() and (ids[:2] == -1).all() and (ids[2, 1:] == -1).all()


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_what_nobody_chose_is_not_read(dtype, mx4):
    layer = Layer(6, 136, 48, dtype, mx4, True, 11)
    x, logits = tokens_of(9, 6, 136, dtype, 12)
    logits[:, 2] = logits[:, 5] = -math.inf
    want = layer.run(x, logits, 3)
    for m in (layer.up, layer.gate, layer.down):
        if mx4:
            m[1][2], m[1][5] = 255, 255
        else:
            m[2], m[5] = math.nan, math.inf
    assert torch.equal(layer.run(x, logits, 3), want)


@pytest.mark.parametrize("mx4", [False, True])
@pytest.mark.parametrize("tokens", [5, 20, 50])
def test_what_is_not_a_number_stays_with_its_token(tokens, mx4):
    layer = Layer(5, 200, 72, torch.float16, mx4, False, 13)
    x, logits = tokens_of(tokens, 5, 200, torch.float16, 14)
    want = layer.run(x, logits, 2)
    x[1, 7], x[tokens - 1, 199] = math.nan, math.inf
    got = layer.run(x, logits, 2)
    touched = [1, tokens - 1]
    rest = [t for t in range(tokens) if t not in touched]
    assert torch.equal(got[rest], want[rest]) and not got[1].isfinite().any()


@pytest.mark.parametrize("up,down", [(2.0 ** 12, 2.0 ** -9), (2.0 ** -40, 2.0 ** 44), (2.0 ** 60, 2.0 ** -64),
                                     (2.0 ** -100, 2.0 ** 100)])
@pytest.mark.parametrize("tokens", [3, 17])
def test_scales_far_from_one(tokens, up, down):
    """4-bit matrices with scales that no bf16 factor of decoding holds."""
    layer = Layer(4, 160, 96, torch.bfloat16, True, False, 15)
    g = generator(16)
    for name, by in (("up", up), ("down", down)):
        w = torch.randn(4, *((96, 160) if name == "up" else (160, 96)), generator=g) * by
        pair = dh.dsmem_mx4_quantize(w.cuda())
        setattr(layer, name, pair)
        setattr(layer, name + "64", stood_for(*pair, w.shape[-1]))
    x, logits = tokens_of(tokens, 4, 160, torch.bfloat16, 17)
    layer.check(layer.run(x, logits, 2), layer.exact(x, logits, 2))


@pytest.mark.parametrize("tokens", [1, 12, 40])
@pytest.mark.parametrize("width,hidden,pad,shift", [(64, 96, 8, 0), (64, 96, 3, 0), (64, 96, 0, 1), (101, 33, 2, 1),
                                                    (128, 64, 16, 8)])
def test_strides_and_odd_bases(tokens, width, hidden, pad, shift):
    layer = Layer(5, width, hidden, torch.bfloat16, False, True, 18)
    x, logits = tokens_of(tokens, 5, width, torch.bfloat16, 19)

    def padded(m):
        base = torch.full((m.numel() // m.shape[-1] * (m.shape[-1] + pad) + shift + 8,), math.nan, dtype=m.dtype,
                          device="cuda")
        view = base[shift:shift + m.numel() // m.shape[-1] * (m.shape[-1] + pad)].view(*m.shape[:-1], -1)
        view[..., :m.shape[-1]] = m
        return view[..., :m.shape[-1]]

    views = [padded(m) for m in (layer.up, layer.gate, layer.down)]
    want = layer.exact(x, logits, 3)
    layer.check(dh.dsmem_expert_layer(padded(x), padded(logits), views[0], views[2], 3, gate=views[1]), want)
    # experts inside rows: [hidden, experts, width] seen as [experts, hidden, width]
    mixed = [m.transpose(0, 1).contiguous().transpose(0, 1) for m in (layer.up, layer.gate, layer.down)]
    layer.check(dh.dsmem_expert_layer(x, logits, mixed[0], mixed[2], 3, gate=mixed[1]), want)


@pytest.mark.parametrize("tokens", [1, 12, 40])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("width,pad,shift", [(128, 3, 0), (128, 0, 1), (101, 2, 1), (256, 8, 8)])
def test_4_bit_matrices_and_tokens_with_odd_bases(width, pad, shift, dtype, tokens):
    layer = Layer(4, width, 72, dtype, True, True, 18)
    x, logits = tokens_of(tokens, 4, width, dtype, 19)
    base = torch.full((tokens * (width + pad) + shift + 8,), math.nan, dtype=dtype, device="cuda")
    view = base[shift:shift + tokens * (width + pad)].view(tokens, -1)[:, :width]
    view.copy_(x)
    layer.check(layer.run(view, logits, 2), layer.exact(x, logits, 2))


@pytest.mark.parametrize("mx4", [False, True])
def test_gate_and_up_may_be_one(mx4):
    layer = Layer(3, 96, 64, torch.bfloat16, mx4, True, 20)
    layer.gate, layer.gate64 = layer.up, layer.up64
    x, logits = tokens_of(6, 3, 96, torch.bfloat16, 21)
    layer.check(layer.run(x, logits, 2, activation="silu"), layer.exact(x, logits, 2, "silu"))


@pytest.mark.parametrize("mx4", [False, True])
def test_matrices_past_32_bits_of_elements(mx4):
    """The last expert's matrices begin behind element 2^32, in the widest rows."""
    experts, width, hidden = 5, 65536, 16400
    g = torch.Generator(device="cuda")
    g.manual_seed(22)

    def make(rows, columns):
        w = torch.randn(rows, columns, generator=g, device="cuda", dtype=torch.bfloat16).div_(math.sqrt(columns))
        if not mx4:
            full = torch.zeros(experts, rows, columns, dtype=torch.bfloat16, device="cuda")
            full[-1] = w
            return full, w
        pair = dh.dsmem_mx4_quantize(w)
        full = tuple(torch.zeros(experts, *t.shape, dtype=torch.uint8, device="cuda") for t in pair)
        for f, t in zip(full, pair):
            f[-1] = t
        return full, dh.dsmem_mx4_dequantize(*pair, columns)

    x = torch.randn(2, width, generator=g, device="cuda", dtype=torch.bfloat16)
    logits = torch.zeros(2, experts, device="cuda")
    logits[:, -1] = 3.0
    up, up_value = make(hidden, width)
    h = torch.relu(torch.stack([torch.mv(up_value[i:i + 4100].double(), t.double()) for t in x
                                for i in range(0, hidden, 4100)]).view(2, hidden))
    del up_value
    down, down_value = make(width, hidden)
    got = dh.dsmem_expert_layer(x, logits, up, down, 1).double()
    want = torch.cat([h @ down_value[i:i + 8192].double().t() for i in range(0, width, 8192)], 1)
    # the output's rounding, and of sums of m terms of either sign about sqrt(m) 2^-24 of the largest
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -12 * want.abs().max()).all()


def guarded(shape, dtype):
    """A tensor of `shape` inside a larger one filled with a pattern, and a check
    that the rest still holds it."""
    n = math.prod(shape)
    raw = torch.full(((n + 512) * dtype.itemsize,), 0x5a, dtype=torch.uint8, device="cuda").view(dtype)
    around, size = raw.view(torch.uint8), dtype.itemsize
    return raw[256:256 + n].view(shape), lambda: bool((around[:256 * size] == 0x5a).all() and (
        around[(256 + n) * size:] == 0x5a).all())


@pytest.mark.parametrize("tokens,width,hidden", [(1, 33, 20), (7, 1000, 70), (33, 129, 8)])
def test_nothing_around_the_answer_is_written(tokens, width, hidden):
    import array
    layer = Layer(4, width, hidden, torch.bfloat16, False, False, 23)
    x, logits = tokens_of(tokens, 4, width, torch.bfloat16, 24)
    want = layer.run(x, logits, 2)
    out, untouched = guarded((tokens, width), torch.bfloat16)
    table = array.array("Q", [layer.up.data_ptr(), 0, width, hidden * width, layer.down.data_ptr(), 0, hidden,
                              hidden * width])
    at = table.buffer_info()[0]
    assert entries._lib.dsmem_expert_layer(
        x.data_ptr(), width, entries.BF16, tokens, width, hidden, logits.data_ptr(), entries.F32, 4, 4, 2, 1, at,
        None, at + 32, 0, out.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out, want) and untouched()


@pytest.mark.parametrize("tokens", [1, 9, 64])
def test_tokens_that_choose_nothing(tokens):
    for mx4 in (False, True):
        layer = Layer(4, 72, 40, torch.float16, mx4, True, 27)
        x, logits = tokens_of(tokens, 4, 72, torch.float16, 28)
        assert (layer.run(x, torch.full_like(logits, -math.inf), 2) == 0).all()


@pytest.mark.parametrize("renormalize", [True, False])
def test_infinite_logits_are_weighted_as_dsmem_route_does(renormalize):
    layer = Layer(6, 64, 48, torch.bfloat16, False, False, 29)
    x, logits = tokens_of(5, 6, 64, torch.bfloat16, 30)
    want = layer.run(x, logits, 2, renormalize=renormalize)
    logits[1, 3] = math.inf
    logits[2, 1] = logits[2, 4] = math.inf
    ids, weights = dh.dsmem_route(logits, 2, renormalize=renormalize)
    got = layer.run(x, logits, 2, renormalize=renormalize)
    exact = few.choices
    try:
        few.choices = lambda *_: (ids.cpu(), weights.cpu())
        y, off = layer.exact(x, logits, 2, renormalize=renormalize)
    finally:
        few.choices = exact
    assert torch.equal(got.isnan().cpu(), y.isnan())
    rest = [t for t in range(5) if not y[t].isnan().any()]
    layer.dtype = got.dtype
    layer.check(got[rest], (y[rest], off[rest]))
    assert torch.equal(got[[0, 3, 4]].isnan(), want[[0, 3, 4]].isnan())


def test_all_of_one_expert():
    """64 tokens of one expert among many: its matrices are passed again."""
    for mx4 in (False, True):
        layer = Layer(9, 136, 200, torch.bfloat16, mx4, True, 31)
        x, logits = tokens_of(64, 9, 136, torch.bfloat16, 32)
        logits[:, 4] = 9.0
        layer.check(layer.run(x, logits, 2), layer.exact(x, logits, 2))


def test_no_tokens():
    layer = Layer(4, 64, 40, torch.bfloat16, False, True, 25)
    x, logits = tokens_of(3, 4, 64, torch.bfloat16, 26)
    assert layer.run(x[:0], logits[:0], 2).shape == (0, 64)


# ---------------------------------------------------------------- 4-bit products

@pytest.mark.parametrize("groups", [1500, 2048])
@pytest.mark.parametrize("outer,out", [(40, torch.float32), (136, torch.bfloat16), (300, torch.float16)])
def test_products_of_many_groups(groups, outer, out):
    g = generator(30)
    sizes = torch.randint(0, 3, (groups,), generator=g)
    n = int(sizes.sum()) + 5
    x, x64 = four_bit(g, n, 200)
    w, w64 = four_bit(g, groups, outer, 200)
    offsets = torch.cat([torch.zeros(1), sizes.cumsum(0)]).to(torch.int32)
    got = dh.dsmem_mx4_grouped_matmul(x, w, offsets.cuda(), out_dtype=out)
    check_product(got, x64, w64, offsets, torch.arange(n))


@pytest.mark.parametrize("inner,shifted", [(32, False), (512, False), (512, True), (70000, False)])
@pytest.mark.parametrize("outer,out", [(33, torch.float32), (36, torch.float32), (17, torch.bfloat16),
                                       (64, torch.float16)])
def test_products_leave_what_is_around_them(inner, shifted, outer, out):
    """Outputs at odd and even bases, values and scales that begin inside others."""
    g = generator(31)
    x, x64 = four_bit(g, 150, inner)
    w, w64 = four_bit(g, 4, outer, inner)
    offsets = torch.tensor([0, 60, 140], dtype=torch.int32)
    x, x64 = tuple(t[1:] for t in x), x64[1:]
    w, w64 = tuple(t[2:] for t in w), w64[2:]
    if shifted:
        x, w = ((v, torch.cat([s.flatten()[:4], s.flatten()])[4:].view(s.shape)) for v, s in (x, w))
    got, untouched = guarded((149, outer), out)
    pitch = w[0].shape[-1] * 2
    dev = offsets.cuda()
    stream = torch.cuda.current_stream().cuda_stream
    assert entries._lib.dsmem_mx4_grouped_matmul(
        x[0].data_ptr(), x[1].data_ptr(), 149, w[0].data_ptr(), w[1].data_ptr(), dev.data_ptr(), 2, None, 1, 149,
        outer, pitch, got.data_ptr(), entries._lib.codes[out], stream) == 0
    check_product(got, x64, w64, offsets, torch.arange(149))
    assert untouched()


def test_products_with_no_rows_to_name():
    g = generator(32)
    w, _ = four_bit(g, 2, 40, 96)
    x, _ = four_bit(g, 3, 96)
    none = tuple(t[:0] for t in x)
    offsets = torch.tensor([0, 2, 4], dtype=torch.int32).cuda()
    order = torch.arange(4, dtype=torch.int32).cuda()
    assert (dh.dsmem_mx4_grouped_matmul(none, w, offsets, order=order) == 0).all()
    assert dh.dsmem_mx4_grouped_matmul(none, w, offsets).shape == (0, 40)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,outer", [(60, 40), (900, 2600), (9000, 2600)])
def test_rows_without_a_source_are_zero_beside_what_is_not_a_number(n, outer, out):
    """Tiles of each width, with NaN in the matrices."""
    g = generator(35)
    x, x64 = four_bit(g, 50, 300)
    w = torch.randn(2, outer, 300, generator=g)
    w[0, ::3, 7] = math.nan
    pair = dh.dsmem_mx4_quantize(w.cuda())
    order = torch.randint(-20, 70, (n,), generator=g).to(torch.int32)
    offsets = torch.tensor([0, n // 2, n - 2], dtype=torch.int32)
    got = dh.dsmem_mx4_grouped_matmul(x, pair, offsets.cuda(), order=order.cuda(), out_dtype=out).cpu()
    there = (order >= 0) & (order < 50) & (torch.arange(n) < n - 2)
    assert (got[~there] == 0).all()
    assert got[: n // 2][there[: n // 2]][:, ::3].isnan().all() and not got[n // 2:].isnan().any()


def test_products_past_32_bits_of_outputs():
    g = generator(33)
    x, x64 = four_bit(g, 64, 32)
    w, w64 = four_bit(g, 2, 65536, 32)
    n = 66000
    order = torch.randint(0, 64, (n,), generator=g).to(torch.int32)
    offsets = torch.tensor([0, 100, n - 3], dtype=torch.int32)
    got = dh.dsmem_mx4_grouped_matmul(x, w, offsets.cuda(), order=order.cuda())
    for p in (0, 99, 100, 65536, 65600, n - 4):
        check_product(got[p:p + 1], x64[order[p]:order[p] + 1], w64[int(p >= 100)][None], torch.tensor([0, 1]),
                      torch.zeros(1, dtype=torch.long))
    assert (got[n - 3:] == 0).all()


@pytest.mark.parametrize("n,outer", [(300, 300), (3000, 1300), (6000, 2600)])
def test_a_wait_that_gives_up_is_reported_by_the_next_call(monkeypatch, n, outer):
    """The copies of a CTA's last stage are withheld, so the wait for them runs out
    with nothing of it in flight (tiles of each width)."""
    g = generator(34)
    x, x64 = four_bit(g, n, 1000)
    w, w64 = four_bit(g, 3, outer, 1000)
    offsets = torch.tensor([0, n // 3, n // 2, n], dtype=torch.int32)
    dev = offsets.cuda()
    want = dh.dsmem_mx4_grouped_matmul(x, w, dev)
    torch.cuda.synchronize()
    monkeypatch.setenv("DSMEM_HIST_TEST_WITHHOLD_LAST_ROUND", "1")
    monkeypatch.setenv("DSMEM_HIST_TEST_WAIT_CYCLES", "200000")
    dh.dsmem_mx4_grouped_matmul(x, w, dev)
    torch.cuda.synchronize()
    monkeypatch.delenv("DSMEM_HIST_TEST_WITHHOLD_LAST_ROUND")
    monkeypatch.delenv("DSMEM_HIST_TEST_WAIT_CYCLES")
    with pytest.raises(dh.DsmemHistError) as e:
        dh.dsmem_mx4_grouped_matmul(x, w, dev)
    assert e.value.code == dh.DSMEM_HIST_ETIMEOUT and "grouped product" in str(e.value)
    assert dh.dsmem_hist_device_status() == 2 and dh.dsmem_hist_device_status() == 0
    assert torch.equal(dh.dsmem_mx4_grouped_matmul(x, w, dev), want)


# ---------------------------------------------------------------- quantisation

def test_the_longest_row():
    from test_gpu_mx4 import quantized
    columns = 2 ** 31 - 513
    x = torch.zeros(1, columns, dtype=torch.bfloat16, device="cuda")
    mark = torch.randn(1, 127, generator=generator(36)).to(torch.bfloat16)
    x[:, -127:] = mark.cuda()
    x[0, 2 ** 30] = -3.0
    values, scales = dh.dsmem_mx4_quantize(x)
    last = columns - columns % 128
    tail = quantized(x[:, last - 128:].cpu())
    assert torch.equal(values[:, last // 2 - 64:].cpu(), tail[0]) and torch.equal(scales[:, last // 32 - 4:].cpu(),
                                                                                 tail[1])
    assert int((scales != 0).sum()) == int((tail[1] != 0).sum()) + 1 and int(scales[0, 2 ** 25]) == 126
    back = dh.dsmem_mx4_dequantize(values, scales, columns, dtype=torch.bfloat16)
    assert float(back[0, 2 ** 30]) == -3.0 and int((back != 0).sum()) <= 128
    want = stood_for(*tail, 128 + columns % 128).to(torch.bfloat16)
    assert torch.equal(back[:, last - 128:].cpu(), want)


# ------------------------------------------------- together, streams, graphs

def four_bit_layer(x, logits, up, down, k):
    """The layer by its parts, in 4 bits throughout."""
    ids, weights = dh.dsmem_route(logits, k)
    offsets, order, position = dh.dsmem_group(ids, up[0].shape[0])
    hidden = dh.dsmem_mx4_grouped_matmul(dh.dsmem_mx4_quantize(x), up, offsets, order=order, fan=k)
    answers = dh.dsmem_mx4_grouped_matmul(dh.dsmem_mx4_quantize(torch.relu(hidden)), down, offsets)
    return dh.dsmem_combine(answers, position.view_as(ids), weights)


def layer_inputs(seed, tokens=40, experts=8, width=256, hidden=136):
    layer = Layer(experts, width, hidden, torch.bfloat16, True, False, seed)
    x, logits = tokens_of(tokens, experts, width, torch.bfloat16, seed + 1)
    return layer, x, logits


def everything(layer, x, logits, k=2):
    up = dh.dsmem_mx4_dequantize(*layer.up, layer.width, dtype=torch.bfloat16)
    down = dh.dsmem_mx4_dequantize(*layer.down, layer.hidden, dtype=torch.bfloat16)
    return (layer.run(x, logits, k), dh.dsmem_expert_layer(x, logits, up, down, k),
            four_bit_layer(x, logits, layer.up, layer.down, k))


def test_the_layer_and_its_parts_agree():
    """4-bit matrices, the same as 16-bit ones, and the parts' products of 4-bit
    rows, whose roundings of x and h are all that differs: each at most a quarter of
    a value, and under an eighth in the mean square."""
    layer, x, logits = layer_inputs(40)
    four, sixteen, parts = everything(layer, x, logits)
    want, off = layer.exact(x, logits, 2)
    layer.check(four, (want, off))
    layer.check(sixteen, (want, off))
    error = (parts.cpu().double() - want).norm() / want.norm()
    assert error < 0.25, float(error)


def test_gradients_through_4_bit_matrices():
    """Products of 4-bit rows forward; backward the 16-bit products of what the
    matrices stand for, against automatic differentiation in 64 bits of a straight
    line through the quantisation."""
    g = generator(41)
    x = torch.randn(90, 192, generator=g).to(torch.bfloat16)
    w = torch.randn(3, 80, 192, generator=g)
    dy = torch.randn(90, 80, generator=g).to(torch.bfloat16)
    offsets = torch.tensor([0, 40, 40, 85], dtype=torch.int32)
    xp, wp = dh.dsmem_mx4_quantize(x.cuda()), dh.dsmem_mx4_quantize(w.cuda())
    x16 = dh.dsmem_mx4_dequantize(*xp, 192, dtype=torch.bfloat16)
    w16 = dh.dsmem_mx4_dequantize(*wp, 192, dtype=torch.bfloat16)
    y = dh.dsmem_mx4_grouped_matmul(xp, wp, offsets.cuda(), out_dtype=torch.float32)
    dx = dh.dsmem_grouped_matmul(dy.cuda(), w16, offsets.cuda(), transpose=True)
    dw = dh.dsmem_grouped_matmul_wgrad(dy.cuda(), x16, offsets.cuda(), out_dtype=torch.float32)
    xd, wd = stood_for(*xp, 192).requires_grad_(), stood_for(*wp, 192).requires_grad_()
    want = torch.zeros(90, 80, dtype=torch.float64)
    for e in range(3):
        a, b = int(offsets[e]), int(offsets[e + 1])
        want = want + torch.cat([torch.zeros(a, 80), xd[a:b] @ wd[e].t(), torch.zeros(90 - b, 80)])
    (want * dy.double()).sum().backward()
    check_product(y, xd.detach(), wd.detach(), offsets, torch.arange(90))
    assert torch.allclose(dx.cpu().double(), xd.grad, rtol=2.0 ** -8, atol=80 * 2.0 ** -23 * 40)
    assert torch.allclose(dw.cpu().double(), wd.grad, rtol=2.0 ** -23, atol=45 * 2.0 ** -23 * 40)


def test_streams_and_threads():
    shapes = [dict(tokens=1), dict(tokens=33, width=264), dict(tokens=64, experts=3, hidden=40),
              dict(tokens=8, experts=200, width=96)]
    inputs = [layer_inputs(50 + j, **s) for j, s in enumerate(shapes)]
    want = [everything(*a) for a in inputs]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    layer, x, logits = inputs[1]
    got = layer.run(x, logits, 2, stream=side)
    values = dh.dsmem_mx4_quantize(x, stream=side)
    back = dh.dsmem_mx4_dequantize(*values, x.shape[1], stream=side)
    side.synchronize()
    assert torch.equal(got, want[1][0]) and torch.equal(back, dh.dsmem_mx4_dequantize(*values, x.shape[1]))
    wrong, start = [], threading.Barrier(4)

    def work(t):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                start.wait()
                for r in range(12):
                    j = (t + r) % len(inputs)
                    got = everything(*inputs[j])
                    stream.synchronize()
                    wrong.extend((t, r, i) for i, (a, b) in enumerate(zip(got, want[j])) if not torch.equal(a, b))
        except Exception as e:  # noqa: BLE001
            wrong.append((t, repr(e)))

    threads = [threading.Thread(target=work, args=(t,)) for t in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not any(t.is_alive() for t in threads) and not wrong, wrong[:3]


def test_two_graphs_in_turn():
    """Captured calls of two layers, replayed in turn, once on two streams at the
    same time, on new contents."""
    inputs = [layer_inputs(60, tokens=1), layer_inputs(61, tokens=24, experts=5)]
    graphs, outs = [], []
    for a in inputs:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            everything(*a)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(everything(*a))
        graphs.append(graph)
    for seed in (70, 80):
        for layer, x, logits in inputs:
            new = tokens_of(x.shape[0], logits.shape[1], x.shape[1], torch.bfloat16, seed)
            x.copy_(new[0])
            logits.copy_(new[1])
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for a, got in zip(inputs, outs):
            for i, (p, q) in enumerate(zip(got, everything(*a))):
                assert torch.equal(p, q), i
        for t in (u for out in outs for u in out):
            t.zero_()
        torch.cuda.synchronize()
        for graph in graphs:
            with torch.cuda.stream(torch.cuda.Stream()):
                graph.replay()
        torch.cuda.synchronize()
        for a, got in zip(inputs, outs):
            for i, (p, q) in enumerate(zip(got, everything(*a))):
                assert torch.equal(p, q), i


def test_scratch_that_cannot_be_had(monkeypatch):
    layer, x, logits = layer_inputs(62)
    want = layer.run(x, logits, 2)
    monkeypatch.setenv("DSMEM_HIST_TEST_FAIL_ALLOC", "1")
    with pytest.raises(dh.DsmemHistError) as e:
        layer.run(x, logits, 2)
    assert e.value.code == dh.DSMEM_HIST_ENOMEM
    monkeypatch.delenv("DSMEM_HIST_TEST_FAIL_ALLOC")
    assert torch.equal(layer.run(x, logits, 2), want)


# ---------------------------------------------------------------- refusals

def test_what_the_python_calls_refuse():
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    logits = torch.ones(4, 3, device="cuda")
    up = torch.ones(3, 40, 64, dtype=torch.bfloat16, device="cuda")
    down = torch.ones(3, 64, 40, dtype=torch.bfloat16, device="cuda")
    up4, down4, x4 = dh.dsmem_mx4_quantize(up), dh.dsmem_mx4_quantize(down), dh.dsmem_mx4_quantize(x)
    off = torch.tensor([0, 2, 3, 4], dtype=torch.int32, device="cuda")
    past = 2 ** 32
    nothing = torch.empty(0, past, dtype=torch.uint8, device="cuda"), torch.empty(0, past // 16, dtype=torch.uint8,
                                                                              device="cuda")
    layer, product = dh.dsmem_expert_layer, dh.dsmem_mx4_grouped_matmul
    for call in [
        lambda: layer(x, logits, up, down, 4), lambda: layer(x, logits, up, down, 0),
        lambda: layer(x, logits, up, down, past + 1), lambda: layer(x, logits, up, down, 1 - past),
        lambda: layer(x, logits[:3], up, down, 1), lambda: layer(x, logits, up, up, 1),
        lambda: layer(x, logits, up[:2], down, 1), lambda: layer(x, logits, up, down, 1, gate=down),
        lambda: layer(x, logits, up, down, 1, activation="gelu"), lambda: layer(x, logits, up, down4, 1),
        lambda: layer(x, logits, up4, down, 1), lambda: layer(x, logits, up4, up4, 1),
        lambda: layer(x, logits, up, down, 1, gate=up4), lambda: layer(x[:, :32], logits, up, down, 1),
        lambda: layer(x.repeat(17, 1), logits.repeat(17, 1), up, down, 1),
        lambda: layer(x, logits, up.transpose(1, 2).contiguous().transpose(1, 2), down, 1),
        lambda: layer(x[:1].expand(4, 64), logits, up, down, 1),
        lambda: layer(x, logits, up[:1].expand(3, 40, 64), down, 1),
        lambda: layer(x, logits, tuple(t[:, :, ::2] for t in up4), down4, 1),
        lambda: product(x4, up4, off[:3]), lambda: product(x4, x4, off),
        lambda: product(x4, up4, off, order=off, fan=past + 1), lambda: product(x4, up4, off, order=off, fan=0),
        lambda: product((x4[0], x4[1][:2]), up4, off), lambda: product((x4[0][:, :32], x4[1]), up4, off),
        lambda: product(tuple(t[::2] for t in x4), up4, off), lambda: product(nothing, up4, off),
        lambda: dh.dsmem_mx4_dequantize(*x4, 0), lambda: dh.dsmem_mx4_dequantize(*x4, 129),
        lambda: dh.dsmem_mx4_dequantize(*nothing, past),
        lambda: dh.dsmem_mx4_quantize(torch.empty(0, past, device="cuda")),
        lambda: dh.dsmem_mx4_quantize(x[:, :0]), lambda: dh.dsmem_mx4_quantize(x.t()),
        lambda: dh.dsmem_mx4_quantize(x[:1].expand(4, 64)),
    ]:
        with pytest.raises((ValueError, dh.DsmemHistError)):
            call()
    for call in [
        lambda: layer(x.float(), logits, up, down, 1), lambda: layer(x.half(), logits, up, down, 1),
        lambda: layer(x, logits.double(), up, down, 1), lambda: layer(x, logits, [], down, 1),
        lambda: layer(x, logits, up, (down4[0],), 1), lambda: layer(x, logits, up, None, 1),
        lambda: product(x, up4, off), lambda: product(x4, up4, off.long()),
        lambda: product(x4, up4, off, out_dtype=torch.float64), lambda: product(x4, up, off),
        lambda: dh.dsmem_mx4_dequantize(*x4, dtype=torch.int32), lambda: dh.dsmem_mx4_dequantize(x, x),
        lambda: dh.dsmem_mx4_quantize(x4[0]),
    ]:
        with pytest.raises(TypeError):
            call()
