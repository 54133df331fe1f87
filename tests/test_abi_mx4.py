"""The 4-bit entries and the whole expert layer without a GPU: what they refuse
before any CUDA call, and calls with nothing to do."""
from __future__ import annotations

import ctypes

import pytest

import cluster_distributed_shared_gb300 as pkg
from test_abi_experts import BF16, F16, F32, P, built, call  # noqa: F401

QUANTIZE = dict(x=P, dtype=BF16, rows=4, columns=100, stride=100, values=P, scales=P, stream=None)
BACK = dict(values=P, scales=P, rows=4, columns=100, dtype=F32, out=P, stream=None)
PRODUCT = dict(x_values=P, x_scales=P, x_rows=4, w_values=P, w_scales=P, offsets=P, groups=2, order=P, fan=2, n=8,
               outer=24, inner=100, out=P, out_dtype=BF16, stream=None)


@pytest.mark.parametrize("name,good,bad", [
    ("dsmem_mx4_quantize", QUANTIZE, bad) for bad in (
        dict(x=None), dict(x=P + 1), dict(dtype=F32, x=P + 2), dict(dtype=3), dict(dtype=-1), dict(rows=-1),
        dict(rows=2 ** 31), dict(columns=0), dict(columns=-5), dict(columns=2 ** 31 - 512, stride=2 ** 31),
        dict(stride=99), dict(stride=0), dict(values=None), dict(values=P + 2), dict(scales=None))] + [
    ("dsmem_mx4_dequantize", BACK, bad) for bad in (
        dict(values=None), dict(values=P + 1), dict(scales=None), dict(rows=-1), dict(rows=2 ** 31),
        dict(columns=0), dict(columns=2 ** 31 - 512), dict(dtype=3), dict(out=None), dict(out=P + 2))] + [
    ("dsmem_mx4_grouped_matmul", PRODUCT, bad) for bad in (
        dict(x_values=None), dict(x_values=P + 8), dict(x_scales=None), dict(x_scales=P + 1), dict(x_rows=-1),
        dict(x_rows=2 ** 31), dict(w_values=None), dict(w_values=P + 4), dict(w_scales=None),
        dict(w_scales=P + 2), dict(offsets=None), dict(offsets=P + 2), dict(groups=0), dict(groups=2049),
        dict(order=P + 2), dict(fan=0), dict(fan=-3), dict(n=-1), dict(n=2 ** 31 - 1), dict(outer=0),
        dict(outer=2 ** 31 - 1), dict(inner=0), dict(inner=2 ** 31 - 512), dict(out=None),
        dict(out=P + 1), dict(out_dtype=F32, out=P + 2), dict(out_dtype=5))])
def test_bad_arguments_are_refused(name, good, bad):
    assert call(name, *dict(good, **bad).values()) == pkg.DSMEM_HIST_EINVAL
    assert pkg.lib().dsmem_hist_last_error()


LAYER = dict(x=P, x_stride=100, dtype=BF16, tokens=4, width=100, hidden=40, logits=P, logits_dtype=F32, experts=8,
             logits_stride=8, top_k=2, renormalize=1, up=(P, 0, 100, 4000), gate=(P, 0, 100, 4000),
             down=(P, 0, 40, 4000), activation=1, out=P, stream=None)
FOUR = dict(up=(P, P, 0, 0), gate=(P, P, 0, 0), down=(P, P, 0, 0))


def layer(args):
    kept = []                                # the tables live until the call is over
    for name in ("up", "gate", "down"):
        if args[name] is not None:
            kept.append((ctypes.c_uint64 * 4)(*args[name]))
            args = dict(args, **{name: ctypes.addressof(kept[-1])})
    return call("dsmem_expert_layer", *args.values())


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=P + 1), dict(x_stride=99), dict(dtype=F32), dict(dtype=7), dict(tokens=-1), dict(tokens=65),
    dict(tokens=2 ** 31 - 1), dict(width=0), dict(width=65537, x_stride=65537), dict(hidden=0), dict(hidden=65537),
    dict(logits=None), dict(logits=P + 2), dict(logits_dtype=4), dict(experts=0), dict(experts=1025,
                                                                                       logits_stride=1025),
    dict(logits_stride=7), dict(top_k=0), dict(top_k=9), dict(experts=64, logits_stride=64, top_k=33),
    dict(up=None), dict(down=None), dict(up=(0, 0, 100, 4000)), dict(up=(P + 1, 0, 100, 4000)),
    dict(up=(P, 0, 99, 4000)), dict(up=(P, 0, 100, 0)), dict(gate=(P, 0, 0, 4000)), dict(down=(P, 0, 39, 4000)),
    dict(down=(P, 0, 40, 2 ** 64 - 4000)), dict(gate=(P, P, 0, 0)), dict(down=(P, P, 0, 0)),
    dict(FOUR, down=(P, 0, 40, 4000)), dict(FOUR, up=(P + 8, P, 0, 0)), dict(FOUR, down=(0, P, 0, 0)),
    dict(activation=2), dict(activation=-1), dict(out=None), dict(out=P + 1)])
def test_bad_layers_are_refused(bad):
    assert layer(dict(LAYER, **bad)) == pkg.DSMEM_HIST_EINVAL
    assert pkg.lib().dsmem_hist_last_error()


def test_nothing_to_do_needs_no_device():
    assert call("dsmem_mx4_quantize", *dict(QUANTIZE, rows=0, x=None).values()) == pkg.DSMEM_HIST_OK
    assert call("dsmem_mx4_dequantize", *dict(BACK, rows=0, out=None).values()) == pkg.DSMEM_HIST_OK
    assert call("dsmem_mx4_grouped_matmul", *dict(PRODUCT, n=0).values()) == pkg.DSMEM_HIST_OK
    assert layer(dict(LAYER, tokens=0, x=None)) == pkg.DSMEM_HIST_OK
    assert layer(dict(LAYER, **FOUR, tokens=0)) == pkg.DSMEM_HIST_OK


def test_cpu_tensors_are_refused():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(3, 64, 64, dtype=torch.bfloat16)
    bytes_ = (torch.zeros(2, 64, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.uint8))
    for run in (lambda: pkg.dsmem_mx4_quantize(x),
                lambda: pkg.dsmem_mx4_quantize([1.0]),
                lambda: pkg.dsmem_mx4_dequantize(*bytes_),
                lambda: pkg.dsmem_mx4_grouped_matmul(bytes_, bytes_, None),
                lambda: pkg.dsmem_mx4_grouped_matmul(x, w, None),
                lambda: pkg.dsmem_expert_layer(x, torch.zeros(2, 3), w, w, 1)):
        with pytest.raises(TypeError):
            run()
