"""The heads' entry points called for the first time in a process inside a stream capture."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROG = """
import torch
from w4a4_quantized_linear_cube_amd import dq
dq.load()
dev = "cuda:0"
pages = 70
zeros = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt, device=dev)
kv = dq.KV(zeros(2 * pages, 2, 16, 64), zeros(2 * pages, 2, 16, 2), zeros(2 * pages, 2, 16, 64), zeros(2 * pages, 2, 16, 2))
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
seqs = dq.Seqs(i32([0, 1, 3]), i32([1000, 500]), torch.arange(2 * pages, dtype=torch.int32, device=dev).view(2, pages))
x = torch.randn(3, 512, device=dev)
table = torch.randn(1100, 32, 2, device=dev)
rope = dq.Rope([table])
qr, out, k, v = (torch.zeros(3, c, device=dev) for c in (256, 256, 128, 128))
a = dq.dq_attn_create(0)

def step():
    dq.dq_kv_write(kv, seqs, x[:, 256:384], x[:, 384:], q=x[:, :256], y=qr, norm="head", rope=rope)
    dq.dq_attn_rows(kv, seqs, qr, a, out)
    dq.dq_kv_read(kv, seqs, k, v)

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    step()
for i in range(3):
    x.copy_(torch.randn(3, 512, generator=torch.Generator().manual_seed(i)))
    seqs.tensors[1].copy_(torch.tensor([1000 + i, 500 + 7 * i], dtype=torch.int32))
    held = [qr, out, k, v, *kv.tensors]
    before = [t.clone() for t in kv.tensors]
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in held]
    for t, b in zip(kv.tensors, before):
        t.copy_(b)
    for t in held[:4]:
        t.fill_(9)
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, held)), i
    assert (out != 0).any() and (out != 9).all()
print("replays agree")
"""


def test_first_call_captured(lib):
    r = subprocess.run([sys.executable, "-c", PROG], capture_output=True, text=True, cwd=ROOT, timeout=100)
    assert r.returncode == 0 and "replays agree" in r.stdout, r.stderr[-2000:]
