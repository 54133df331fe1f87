"""Sizes at the ends of the expert-layer entry points' ranges, without a GPU:
what the kernels' 32-bit index arithmetic cannot hold is refused before any
CUDA call."""
from __future__ import annotations

import pytest

import cluster_distributed_shared_gb300 as pkg
from test_abi_experts import COMBACK, COMBINE, MATMUL, WGRAD, built, call  # noqa: F401

WIDEST = 2 ** 31 - 2049
LONGEST = 2 ** 31 - 513


@pytest.mark.parametrize("name,good,bad", [
    ("dsmem_combine", COMBINE, dict(width=WIDEST + 1, z_stride=WIDEST + 1)),
    ("dsmem_combine", COMBINE, dict(width=2 ** 31 - 1, z_stride=2 ** 31)),
    ("dsmem_combine_backward", COMBACK, dict(width=WIDEST + 1, z_stride=2 ** 31, dy_stride=2 ** 31)),
    ("dsmem_grouped_matmul", MATMUL, dict(inner=LONGEST + 1, x_stride=2 ** 31, weight_row_stride=2 ** 31)),
    ("dsmem_grouped_matmul", MATMUL, dict(outer=2 ** 31 - 1)),
    ("dsmem_grouped_matmul_wgrad", WGRAD, dict(inner=2 ** 31 - 1, x_stride=2 ** 31)),
    ("dsmem_grouped_matmul_wgrad", WGRAD, dict(outer=LONGEST + 1, dy_stride=2 ** 31)),
])
def test_sizes_past_the_index_arithmetic_are_refused(name, good, bad):
    assert call(name, *dict(good, **bad).values()) == pkg.DSMEM_HIST_EINVAL
