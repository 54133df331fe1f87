"""The expert-layer entry points without a GPU: declared, exported, and refusing
bad arguments before any CUDA call."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

import cluster_distributed_shared_gb300 as pkg
from cluster_distributed_shared_gb300 import experts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x1000          # an aligned address that is never read: every call here is refused
F32, F16, BF16 = experts.F32, experts.F16, experts.BF16


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def call(name, *args):
    fn = getattr(pkg.lib(), name)
    fn.argtypes = experts.SIGNATURES[name]
    fn.restype = ctypes.c_int
    return fn(*args)


def test_header_is_c(tmp_path):
    source = tmp_path / "c.c"
    source.write_text('#include "dsmem_experts.h"\nint main(void) { return DSMEM_BF16 - 2; }\n')
    cuda = os.path.join(os.path.dirname(os.path.dirname(__import__(
        "cluster_distributed_shared_gb300._build", fromlist=["nvcc"]).nvcc())), "include")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                    "-I", cuda, "-c", str(source), "-o", str(tmp_path / "c.o")], check=True)


def test_signatures_name_exported_functions():
    assert set(experts.SIGNATURES) <= set(pkg.EXPORTS)
    for name in experts.SIGNATURES:
        assert hasattr(pkg.lib(), name) and callable(getattr(pkg, name))


ROUTE = dict(logits=P, dtype=F32, tokens=4, experts=8, row_stride=8, top_k=2, renormalize=1, ids=P,
             weights=P, stream=None)
BACK = dict(logits=P, dtype=F32, tokens=4, experts=8, row_stride=8, top_k=2, renormalize=1, ids=P,
            weights=P, grad_weights=P, grad_logits=P, stream=None)
GROUP = dict(keys=P, n=4, num_groups=8, offsets=P, order=P, position=P, stream=None)
MATMUL = dict(x=P, x_rows=4, x_stride=16, weight=P, weight_row_stride=16, weight_group_stride=128,
              offsets=P, groups=2, order=P, fan=1, n=4, outer=8, inner=16, transpose=0, dtype=BF16, out=P,
              out_dtype=BF16, stream=None)
WGRAD = dict(dy=P, dy_stride=8, x=P, x_rows=4, x_stride=16, offsets=P, groups=2, order=P, fan=1, n=4,
             outer=8, inner=16, dtype=BF16, out=P, out_dtype=BF16, stream=None)
COMBINE = dict(z=P, z_rows=8, z_stride=16, position=P, weights=P, tokens=4, top_k=2, width=16, dtype=F16,
               out=P, stream=None)
COMBACK = dict(dy=P, dy_stride=16, z=P, z_stride=16, position=P, order=P, weights=P, tokens=4, top_k=2,
               width=16, dtype=F16, dz=P, dweights=P, stream=None)


@pytest.mark.parametrize("name,good,bad", [
    ("dsmem_route", ROUTE, dict(logits=None)), ("dsmem_route", ROUTE, dict(logits=P + 2)),
    ("dsmem_route", ROUTE, dict(dtype=3)), ("dsmem_route", ROUTE, dict(tokens=-1)),
    ("dsmem_route", ROUTE, dict(tokens=2 ** 31)), ("dsmem_route", ROUTE, dict(experts=0)),
    ("dsmem_route", ROUTE, dict(experts=1025, row_stride=1025)), ("dsmem_route", ROUTE, dict(top_k=9)),
    ("dsmem_route", ROUTE, dict(top_k=0)), ("dsmem_route", ROUTE, dict(row_stride=7)),
    ("dsmem_route", ROUTE, dict(ids=None)), ("dsmem_route", ROUTE, dict(weights=P + 1)),
    ("dsmem_route_backward", BACK, dict(grad_weights=None)),
    ("dsmem_route_backward", BACK, dict(grad_logits=P + 2)), ("dsmem_route_backward", BACK, dict(top_k=33)),
    ("dsmem_group", GROUP, dict(n=-1)), ("dsmem_group", GROUP, dict(n=2 ** 31)),
    ("dsmem_group", GROUP, dict(num_groups=0)), ("dsmem_group", GROUP, dict(num_groups=32769)),
    ("dsmem_group", GROUP, dict(keys=None)), ("dsmem_group", GROUP, dict(offsets=P + 2)),
    ("dsmem_grouped_matmul", MATMUL, dict(dtype=F32)), ("dsmem_grouped_matmul", MATMUL, dict(out_dtype=F16)),
    ("dsmem_grouped_matmul", MATMUL, dict(groups=0)), ("dsmem_grouped_matmul", MATMUL, dict(groups=2049)),
    ("dsmem_grouped_matmul", MATMUL, dict(fan=0)), ("dsmem_grouped_matmul", MATMUL, dict(n=2 ** 31 - 1)),
    ("dsmem_grouped_matmul", MATMUL, dict(x_stride=15)), ("dsmem_grouped_matmul", MATMUL, dict(outer=0)),
    ("dsmem_grouped_matmul", MATMUL, dict(weight_row_stride=8)),
    ("dsmem_grouped_matmul", MATMUL, dict(weight_group_stride=0)),
    ("dsmem_grouped_matmul", MATMUL, dict(x=P + 1)), ("dsmem_grouped_matmul", MATMUL, dict(weight=None)),
    ("dsmem_grouped_matmul", MATMUL, dict(offsets=None)), ("dsmem_grouped_matmul", MATMUL, dict(order=P + 2)),
    ("dsmem_grouped_matmul", MATMUL, dict(transpose=1, x_stride=7)),
    ("dsmem_grouped_matmul_wgrad", WGRAD, dict(dy_stride=7)),
    ("dsmem_grouped_matmul_wgrad", WGRAD, dict(dy=None)), ("dsmem_grouped_matmul_wgrad", WGRAD, dict(out=None)),
    ("dsmem_grouped_matmul_wgrad", WGRAD, dict(inner=0)),
    ("dsmem_combine", COMBINE, dict(z_stride=15)), ("dsmem_combine", COMBINE, dict(top_k=0)),
    ("dsmem_combine", COMBINE, dict(tokens=2 ** 30)), ("dsmem_combine", COMBINE, dict(position=None)),
    ("dsmem_combine", COMBINE, dict(weights=P + 2)), ("dsmem_combine", COMBINE, dict(dtype=-1)),
    ("dsmem_combine_backward", COMBACK, dict(order=None)),
    ("dsmem_combine_backward", COMBACK, dict(weights=None)),
    ("dsmem_combine_backward", COMBACK, dict(dy_stride=3)),
])
def test_bad_arguments_are_refused(name, good, bad):
    args = dict(good, **bad)
    assert call(name, *args.values()) == pkg.DSMEM_HIST_EINVAL
    assert pkg.lib().dsmem_hist_last_error()


def entry(grad=P, out=P, count=4, dtype=F32):
    return [grad or 0, out or 0, count, dtype & 0xFFFFFFFF]


@pytest.mark.parametrize("words,max_norm,norm", [
    (entry(), 0.0, P), (entry(), float("nan"), P), (entry(), float("inf"), P), (entry(), 1.0, None),
    (entry(dtype=7), 1.0, P), (entry(grad=None), 1.0, P), (entry(out=P + 2), 1.0, P),
    (entry(count=2 ** 63), 1.0, P), (entry(count=2 ** 50), 1.0, P)])
def test_bad_gradients_are_refused(words, max_norm, norm):
    table = (ctypes.c_uint64 * 4)(*words)
    assert call("dsmem_grad_clip", table, 1, max_norm, norm, None) == pkg.DSMEM_HIST_EINVAL


def test_nothing_to_do_needs_no_device():
    assert call("dsmem_route", *dict(ROUTE, tokens=0).values()) == pkg.DSMEM_HIST_OK
    assert call("dsmem_combine", *dict(COMBINE, tokens=0).values()) == pkg.DSMEM_HIST_OK
    assert call("dsmem_grouped_matmul", *dict(MATMUL, n=0).values()) == pkg.DSMEM_HIST_OK


def test_cpu_tensors_are_refused():
    torch = pytest.importorskip("torch")
    for run in (lambda: pkg.dsmem_route(torch.zeros(2, 4), 2),
                lambda: pkg.dsmem_group(torch.zeros(2, dtype=torch.int32), 2),
                lambda: pkg.dsmem_grouped_matmul(torch.zeros(2, 8), torch.zeros(1, 8, 8), None),
                lambda: pkg.dsmem_combine(torch.zeros(2, 8), torch.zeros(1, 2, dtype=torch.int32)),
                lambda: pkg.dsmem_grad_clip([torch.zeros(2)], 1.0)):
        with pytest.raises(TypeError):
            run()
