"""Few-row operators without a GPU: every refusal of the C entry points and
of the binding, and the oracle they are compared with."""
import ctypes
import math
import os
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from oracle import mx, rows
from w4a4_quantized_linear_cube_amd import dq

INTERNAL = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "w4a4_quantized_linear_cube_amd", "csrc",
                        "dq_internal.h")
A16 = 1 << 20            # an address that is never followed: every call below is refused first


def _norm(lib, **kw):
    a = dict(x=A16, ldx=64, r=None, ldr=0, dt=1, g=None, gdt=0, eps=1e-6, N=4, C=64, group=32, h=None, ldh=0, codes=2 * A16,
             scales=3 * A16, y=None, ldy=0, device=0)
    a.update(kw)
    return lib.dq_rmsnorm8(a["x"], a["ldx"], a["r"], a["ldr"], a["dt"], a["g"], a["gdt"], a["eps"], a["N"], a["C"], a["group"],
                           a["h"], a["ldh"], a["codes"], a["scales"], a["y"], a["ldy"], a["device"], None)


@pytest.mark.parametrize("status,kw", [
    (1, dict(dt=2)), (1, dict(g=A16, gdt=5)), (1, dict(group=16)), (2, dict(group=64, C=96, ldx=96)),
    (1, dict(eps=0.0)), (1, dict(eps=-1.0)), (1, dict(eps=math.nan)), (1, dict(eps=math.inf)), (1, dict(eps=1e-61)),
    (2, dict(C=48)), (2, dict(C=0)), (2, dict(C=32768 + 32, ldx=32768 + 32)), (2, dict(N=-1)), (2, dict(N=2 ** 31)),
    (1, dict(codes=None)), (1, dict(scales=None)), (1, dict(codes=None, scales=None)), (1, dict(x=None)),
    (1, dict(h=5 * A16, ldh=64)),                                       # h without a residual
    (2, dict(ldx=63)), (2, dict(ldx=68)), (2, dict(ldx=2 ** 50)), (1, dict(x=A16 + 8)), (1, dict(g=A16 + 4)),
    (1, dict(codes=2 * A16 + 4)), (2, dict(r=A16, ldr=32)), (1, dict(y=5 * A16 + 2, ldy=64)),
    (1, dict(r=4 * A16, ldr=64, h=A16 + 128, ldh=64)),                  # h one row behind x
    (1, dict(r=4 * A16, ldr=64, h=A16, ldh=72)),                        # x's memory at another stride
    (1, dict(y=A16 + 64, ldy=64, N=1)),                                 # half a row behind x
    (1, dict(r=4 * A16, ldr=64, h=5 * A16, ldh=64, y=5 * A16, ldy=64)),
    (1, dict(ldx=192, y=A16 + 64, ldy=192)),                            # overlapping columns of one wide buffer
    (1, dict(ldx=192, y=A16 - 64, ldy=192)),                            # the same from below
    (1, dict(ldx=192, y=A16 + 192 * 2 - 16, ldy=192)),                  # one row on, less 8 columns
    (1, dict(codes=A16)), (1, dict(scales=A16 + 511)), (1, dict(codes=2 * A16, scales=2 * A16 + 255)),
    (1, dict(g=A16 * 2 + 240, gdt=0)), (1, dict(y=2 * A16 + 16, ldy=64)), (1, dict(g=5 * A16, gdt=1, y=5 * A16 - 368, ldy=64)),
])
def test_norm_refusals(lib, status, kw):
    assert _norm(lib, **kw) == status, lib.dq_last_error().decode()
    assert lib.dq_last_error().decode()


def test_overlap_rule_against_brute_force(tmp_path):
    """The rule that the refusals use, on small arrays: bytes that both hold, by
    listing them; equal pitches exactly, unequal ones by their ranges."""
    import shutil
    import subprocess
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    src = open(INTERNAL).read()
    body = src[src.index("struct Span {"):src.index("// Makes a handle's device current")]
    prog = tmp_path / "overlap.cpp"
    prog.write_text("#include <cstdint>\n#include <cstdio>\n#include <set>\n" + body + """
int main() {
    long bad = 0, n = 0;
    char* base = (char*)4096;
    for (long pa = 1; pa <= 7; ++pa) for (long wa = 1; wa <= pa; ++wa) for (long pb = pa; pb <= pa + 1; ++pb)
    for (long wb = 1; wb <= pb; ++wb) for (long at = -24; at <= 24; ++at) for (long ra = 1; ra <= 3; ++ra) for (long rb = 1; rb <= 3; ++rb) {
        std::set<long> held;
        for (long r = 0; r < ra; ++r) for (long c = 0; c < wa; ++c) held.insert(r * pa + c);
        bool real = false;
        for (long r = 0; r < rb; ++r) for (long c = 0; c < wb; ++c) real |= held.count(at + r * pb + c) > 0;
        const bool said = overlap(Span{base, ra, pa, wa}, Span{base + at, rb, pb, wb});
        const bool ranges = at < (ra - 1) * pa + wa && at + (rb - 1) * pb + wb > 0;
        const bool back = overlap(Span{base + at, rb, pb, wb}, Span{base, ra, pa, wa});
        if ((real && !said) || said != back || (said && !ranges)) ++bad;             // never missed, the same both ways
        if (pa == pb && ra == rb && ra > 1 && said && !real && ranges) {             // slices side by side are let through
            const long d = ((at % pa) + pa) % pa;
            if (d >= wa && d + wb <= pa) ++bad;
        }
        ++n;
    }
    printf("%ld of %ld wrong\\n", bad, n);
    return bad != 0;
}
""")
    exe = tmp_path / "overlap"
    subprocess.run(["g++", "-std=c++17", "-O1", str(prog), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


def test_norm_of_no_rows(lib):
    assert _norm(lib, N=0) == 0
    assert _norm(lib, N=0, x=None) == 0


def test_row_product_refusals(lib):
    h = ctypes.c_void_p()
    assert lib.dq_rows_create(None, 4, ctypes.byref(h)) == 1
    assert lib.dq_rows_create(None, 4, None) == 1
    assert lib.dq_linear_rows(None, A16, 1, 64, 1, None, A16, 0, 64, None) == 1
    assert lib.dq_linear_rows8(None, A16, A16, 1, None, A16, 0, 64, None) == 1
    lib.dq_rows_destroy(None)


def test_import_refusals(lib):
    codes, scales = np.zeros((64, 48), np.uint8), np.full((64, 3), 127, np.uint8)
    l1, l2 = np.zeros((96, 8), np.uint16), np.zeros((8, 64), np.uint16)
    h = ctypes.c_void_p()
    P = lambda a: None if a is None else ctypes.c_void_p(a.ctypes.data)
    call = lambda c=codes, s=scales, ci=96, co=64, rank=8, a=l1, b=l2: lib.dq_import_weights(
        P(c), P(s), ci, co, rank, P(a), P(b), 0, ctypes.byref(h))
    assert call(c=None) == 1 and call(s=None) == 1 and call(a=None) == 1 and call(b=None) == 1
    assert call(ci=80) == 2 and call(ci=0) == 2 and call(co=0) == 2 and call(co=2 ** 25) == 2
    assert call(rank=-1) == 1 and call(rank=65) == 1
    bad = scales.copy()
    bad[63, 2] = 255
    assert call(s=bad) == 1 and "255" in lib.dq_last_error().decode()
    assert not h.value


W = SimpleNamespace(Ci=64, Co=96, rank=16, device=0, handle=None)
R = SimpleNamespace(weights=W, handle=None, max_rows=8, pair=None)


def _raises(fn, *args, match, **kw):
    with pytest.raises(dq.DQError, match=match):
        fn(*args, **kw)


def test_binding_refusals(lib):
    y = torch.zeros(3, 96)
    f = dq.dq_linear_rows
    _raises(f, W, torch.zeros(3, 64, dtype=torch.float16), R, y, match="dtype")
    _raises(f, W, torch.zeros(3, 32), R, y, match="shape")
    _raises(f, W, torch.zeros(64), R, y, match="shape")
    _raises(f, W, torch.zeros(64, 3).t(), R, y, match="contiguous, non-overlapping")
    _raises(f, W, torch.zeros(1, 64).expand(3, 64), R, y, match="contiguous, non-overlapping")
    _raises(f, W, np.zeros((3, 64), np.float32), R, y, match="torch tensor")
    _raises(f, W, torch.zeros(3, 64), R, y, match="cuda:0")
    _raises(f, SimpleNamespace(Ci=64, Co=32, rank=16, device=0, handle=None), torch.zeros(3, 64), R, y, match="different weight")
    f = dq.dq_linear_rows8
    _raises(f, W, torch.zeros(3, 64, dtype=torch.int8), torch.zeros(3, 2, dtype=torch.uint8), R, y, match="dtype")
    _raises(f, W, torch.zeros(3, 128, dtype=torch.uint8)[:, :64], torch.zeros(3, 2, dtype=torch.uint8), R, y, match="contiguous")
    f = dq.dq_rmsnorm8
    _raises(f, torch.zeros(3, 64), None, 1e-6, match="on a GPU")
    _raises(f, np.zeros((3, 64)), None, 1e-6, match="on a GPU")
    f = dq.dq_import_weights
    c, s = np.zeros((96, 32), np.uint8), np.zeros((96, 2), np.uint8)
    _raises(f, c.astype(np.int8), s, None, None, match="uint8")
    _raises(f, c, s[:, :1], None, None, match="rscales has shape")
    _raises(f, c, s, np.zeros((64, 4), np.uint16), None, match="both factors")
    _raises(f, c, s, np.zeros((63, 4), np.uint16), np.zeros((4, 96), np.uint16), match="l1 has shape")


# ---- the oracle --------------------------------------------------------------
def test_oracle_norm_by_scalars():
    """Every step again for one row, one element at a time."""
    rng = np.random.default_rng(5)
    x = rows.to_stream(rng.standard_normal((1, 64)) * 3, "bf16")
    r = rows.to_stream(rng.standard_normal((1, 64)), "bf16")
    g = rng.standard_normal(64).astype(np.float32)
    got = rows.rms_norm8(x, r, g, 1e-5, "bf16")
    s, h = 0.0, []
    for c in range(64):
        bits = int(np.float32(x[0, c] + r[0, c]).view(np.uint32))
        kept = (bits + 0x7FFF + (bits >> 16 & 1)) >> 16 << 16
        h.append(np.uint32(kept & 0xFFFFFFFF).view(np.float32))
        s += float(h[-1]) ** 2
    f = np.float32(1.0 / math.sqrt(s / 64 + 1e-5))
    for G in range(2):
        v = [np.float32(np.float32(h[c] * f) * g[c]) for c in range(32 * G, 32 * G + 32)]
        e = -127
        while max(abs(float(t)) for t in v) > 448.0 * 2.0 ** e:
            e += 1
        assert got["scales"][0, G] == e + 127
        for i, t in enumerate(v):
            grid = [mx.fp8_decode_magnitude(k) for k in range(127)]
            want = min(range(127), key=lambda k: (abs(grid[k] - abs(float(t)) / 2.0 ** e), k % 2))
            assert got["codes"][0, 32 * G + i] == want | (128 if np.signbit(t) else 0)
    assert np.array_equal(got["h"][0], np.array(h))


def test_oracle_norm_is_scale_free_and_groups_share():
    x = np.random.default_rng(6).standard_normal((3, 128)).astype(np.float32)
    a, b = rows.rms_norm8(x, None, None, 1e-60, "f32"), rows.rms_norm8(4 * x, None, None, 1e-60, "f32")
    assert np.array_equal(a["codes"], b["codes"]) and np.array_equal(a["scales"], b["scales"])
    w = rows.rms_norm8(x, None, None, 1e-60, "f32", group=64)
    assert np.array_equal(w["scales"][:, 0::2], w["scales"][:, 1::2])
    assert np.array_equal(w["scales"][:, 0::2], np.maximum(a["scales"][:, 0::2], a["scales"][:, 1::2]))
    assert abs(float((a["v"].astype(np.float64) ** 2).mean()) - 1.0) < 1e-6


def test_oracle_product_is_the_dense_one():
    rng = np.random.default_rng(7)
    rc, rs = rng.integers(0, 256, (40, 32), dtype=np.uint8), rng.integers(120, 130, (40, 2), dtype=np.uint8)
    l1 = mx.f32_to_bf16_bits(rng.standard_normal((64, 3)).astype(np.float32))
    l2 = mx.f32_to_bf16_bits(rng.standard_normal((3, 40)).astype(np.float32))
    x = rng.standard_normal((5, 64))
    grid = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    dense = np.zeros((64, 40))
    for j in range(40):
        for c in range(64):
            k = int(rc[j, c // 2]) >> (4 * (c % 2)) & 15
            dense[c, j] = (-1) ** (k >> 3) * grid[k & 7] * 2.0 ** (int(rs[j, c // 32]) - 127)
    dense += mx.bf16_bits_to_f64(l1) @ mx.bf16_bits_to_f64(l2)
    y, main, low = rows.product(x, rc, rs, l1, l2)
    np.testing.assert_allclose(y, x @ dense, rtol=0, atol=1e-12 * float((main + low).max()))
    assert (np.abs(y) <= (main + low) * (1 + 1e-12)).all()


def test_binding_names_its_calls():
    """Every status that the binding checks is checked under one function's name."""
    import ast
    import inspect
    tree = ast.parse(inspect.getsource(dq))
    calls = [c for c in ast.walk(tree) if isinstance(c, ast.Call) and isinstance(c.func, ast.Name) and c.func.id == "_check"]
    assert len(calls) > 30
    for c in calls:
        assert len(c.args) == 2 and not c.keywords, ast.unparse(c)
        if isinstance(c.args[1], ast.Constant):
            assert c.args[1].value in dq.EXPORTS, ast.unparse(c)


def test_one_hip_runtime():
    """The library loaded first, torch after it: both use one HIP runtime (with
    two, neither knows the other's streams and memory)."""
    import subprocess
    import sys
    prog = ("from w4a4_quantized_linear_cube_amd import dq; dq.load(); import torch; "
            "print(len({l.split()[-1] for l in open('/proc/self/maps') if 'libamdhip64' in l}))")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", prog], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split()[-1] == "1", r.stdout
