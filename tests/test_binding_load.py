"""What loading the library needs: libdq.so alone.  The native marshalling of
the small calls and torch serve it where they are there."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "w4a4_quantized_linear_cube_amd"

PROG = """
import sys, warnings
if {blocked!r}:
    sys.modules[{blocked!r}] = None               # importing it raises ImportError
from w4a4_quantized_linear_cube_amd import dq
with warnings.catch_warnings(record=True) as said:
    warnings.simplefilter("always")
    lib = dq.load()
    assert dq.load() is lib
assert lib.dq_status_str(1).decode(), "an entry point answers"
assert lib.dq_linear_rows(None, None, 0, 0, 0, None, None, 0, 0, None) == 1
print(len([w for w in said if "_dqcall" in str(w.message) and "build" in str(w.message)]), dq._CALL is None)
"""


@pytest.mark.parametrize("blocked,native,warned", [("", "absent", 1), ("", "broken", 1), ("torch", "absent", 0), ("torch", "built", 0),
                                                   ("", "built", 0)])
def test_load_needs_only_the_library(lib, tmp_path, blocked, native, warned):
    """Without _dqcall.so, with one that cannot be loaded, and without torch,
    load() gives the library; where torch's users lose the native marshalling by
    that, it says so once, and what to run."""
    here, src = tmp_path / PACKAGE, os.path.join(ROOT, PACKAGE)
    here.mkdir()
    for name in os.listdir(src):
        if name.endswith(".py"):
            shutil.copy(os.path.join(src, name), here / name)
    os.symlink(os.path.join(src, "libdq.so"), here / "libdq.so")
    if native == "built":
        if not os.path.exists(os.path.join(src, "_dqcall.so")):
            pytest.skip("_dqcall.so is not built")
        shutil.copy(os.path.join(src, "_dqcall.so"), here / "_dqcall.so")
    elif native == "broken":
        (here / "_dqcall.so").write_bytes(b"not a library")
    r = subprocess.run([sys.executable, "-c", PROG.format(blocked=blocked)], capture_output=True, text=True, cwd=tmp_path, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split() == [str(warned), str(bool(warned or blocked))], r.stdout


def test_refusals_without_the_native_part(lib, monkeypatch):
    import torch
    from types import SimpleNamespace
    from w4a4_quantized_linear_cube_amd import dq
    monkeypatch.setattr(dq, "_CALL", None)
    w = SimpleNamespace(Ci=64, Co=96, rank=16, device=0, handle=None)
    a = SimpleNamespace(weights=w, handle=None, max_rows=8, pair=None)
    with pytest.raises(dq.DQError, match="on a GPU"):
        dq.dq_rmsnorm8(torch.zeros(3, 64), None, 1e-6)
    with pytest.raises(dq.DQError, match="cuda:0"):
        dq.dq_linear_rows(w, torch.zeros(3, 64), a, torch.zeros(3, 96))
    with pytest.raises(dq.DQError, match="cuda:0"):
        dq.dq_linear_rows8(w, torch.zeros(3, 64, dtype=torch.uint8), torch.zeros(3, 2, dtype=torch.uint8), a, torch.zeros(3, 96))


@pytest.mark.gpu
@pytest.mark.parametrize("n", [0, 1, 5])
def test_both_ways_of_marshalling_agree(lib, monkeypatch, n):
    """The same calls through _dqcall.so and through the checks of the binding
    itself, strided rows and every optional argument among them."""
    import numpy as np
    import torch
    from w4a4_quantized_linear_cube_amd import dq
    assert dq._CALL is not None
    rng = np.random.default_rng(n)
    ci, co, dev = 160, 72, "cuda:0"
    w = dq.dq_import_weights(rng.integers(0, 256, (co, ci // 2), dtype=np.uint8), rng.integers(119, 127, (co, ci // 32), dtype=np.uint8),
                             None, None)
    a = dq.dq_rows_create(w, 8)
    x = torch.randn(n, ci + 16, generator=torch.Generator().manual_seed(n)).to(dev)[:, 8:8 + ci]
    gain = torch.linspace(0.5, 2.0, ci, device=dev)

    def step(stream):
        codes, scales = (torch.full((n, k), 7, dtype=torch.uint8, device=dev) for k in (ci, ci // 32))
        h, plain = (torch.zeros(n, ci, device=dev) for _ in range(2))
        wide = torch.zeros(n, co + 8, device=dev)
        y8 = torch.zeros(n, co, dtype=torch.bfloat16, device=dev)
        dq.dq_rmsnorm8(x, gain, 1e-5, codes, scales, residual=x, h=h, y=plain, stream=stream)
        dq.dq_linear_rows(w, x, a, wide[:, 3:3 + co], stream)
        dq.dq_linear_rows8(w, codes, scales, a, y8, stream)
        dq.dq_rmsnorm8(x, None, 1e-5, codes, scales, stream=stream)
        torch.cuda.synchronize()
        return codes, scales, h, plain, wide, y8

    for stream in (None, torch.cuda.current_stream(), torch.cuda.current_stream().cuda_stream):
        with monkeypatch.context() as m:
            native = step(stream)
            m.setattr(dq, "_CALL", None)
            assert all(torch.equal(p, q) for p, q in zip(native, step(stream)))
