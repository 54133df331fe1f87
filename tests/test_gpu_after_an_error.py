"""A call that the runtime refuses leaves no error behind for the next call."""
from __future__ import annotations

import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# dsmem_hist_device_status copies on the default stream, which the runtime refuses while
# a stream that waits for the default one is captured (and the capture is then over).
# Driver calls make the stream and begin and end the capture, so that torch's own
# state has no part in it.
CHILD = """
import ctypes
import sys
sys.path.insert(0, {root!r})
import torch
import cluster_distributed_shared_gb300 as dh

x = torch.randn(8, 256, device="cuda")
logits = torch.randn(8, 4, device="cuda")
calls = [lambda: dh.dsmem_mx4_quantize(x)[0], lambda: dh.dsmem_route(logits, 2)[0],
         lambda: dh.dsmem_hist(torch.arange(1000, dtype=torch.int32, device="cuda"), 1000)]
want = [call() for call in calls]
torch.cuda.synchronize()
driver = ctypes.CDLL("libcuda.so.1")
handle = ctypes.c_void_p()
assert driver.cuStreamCreate(ctypes.byref(handle), 0) == 0
for call, right in zip(calls, want):
    assert driver.cuStreamBeginCapture_v2(handle, 0) == 0
    try:
        dh.dsmem_hist_device_status()
        refused = False
    except dh.DsmemHistError as e:
        refused = e.code == dh.DSMEM_HIST_ECUDA
    graph = ctypes.c_void_p()
    driver.cuStreamEndCapture(handle, ctypes.byref(graph))
    assert refused
    got = call()
    torch.cuda.synchronize()
    assert torch.equal(got, right)
print("ok")
"""


def test_a_refused_call_leaves_nothing_for_the_next():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    r = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr
