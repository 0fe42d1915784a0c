"""The library's first launch of a process inside a stream capture: nothing was
called before that could have loaded a kernel or asked for the device."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROG = """
import sys
import numpy as np
import torch
from w4a4_quantized_linear_cube_amd import dq
dq.load()
n, c, co, dev = 3, 512, 300, "cuda:0"
x = torch.randn(n, c, device=dev)
codes, scales = (torch.zeros(n, k, dtype=torch.uint8, device=dev) for k in (c, c // 32))
y = torch.zeros(n, co, device=dev)
if {product}:
    rng = np.random.default_rng(1)
    w = dq.dq_import_weights(rng.integers(0, 256, (co, c // 2), dtype=np.uint8), rng.integers(119, 127, (co, c // 32), dtype=np.uint8), None, None)
    a = dq.dq_rows_create(w, n)

def step():
    dq.dq_rmsnorm8(x, None, 1e-6, codes, scales)
    if {product}:
        dq.dq_linear_rows8(w, codes, scales, a, y)

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
for i in range(3):
    x.copy_(torch.randn(n, c, generator=torch.Generator().manual_seed(i)))
    codes.fill_(9), y.fill_(9)
    graph.replay()
    torch.cuda.synchronize()
    got = codes.clone(), scales.clone(), y.clone()
    codes.fill_(9), scales.fill_(9), y.fill_(9)
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, (codes, scales, y))), i
    assert (codes != 9).any()
print("replays agree")
"""


@pytest.mark.parametrize("product", [False, True])
def test_first_call_captured(lib, product):
    r = subprocess.run([sys.executable, "-c", PROG.format(product=product)], capture_output=True, text=True, cwd=ROOT, timeout=100)
    assert r.returncode == 0 and "replays agree" in r.stdout, r.stderr[-2000:]
