"""Few-row products (dq_linear_rows, dq_linear_rows8) and imported weights on
the GPU against the oracle.

Two kinds of comparison:
  * inputs whose products and sums are all exact in fp32 (small integers
    times powers of two): every output equal, whatever the order of sums, so
    a channel, row or scale taken wrongly shows;
  * random inputs, within the bound of fp32 sums in any order.  Products are
    exact (2-bit weights times at most 24-bit values in 8-bit parts), each of
    the k additions behind an output is off by at most 2^-24 of the sum of
    its terms' magnitudes M (2^-23 where the instruction truncates), so
    |error| <= k 2^-23 M with k = parts Ci + 8 for the main sum (a share of it
    per wave, then the shares) and parts Ci + 2 rank + 8 for the low-rank one;
    plus half a step of y's type.
"""
import numpy as np
import pytest
import torch

from oracle import mx, rows
from parity_util import DEV, _random_factors, _say

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def dqm(lib):
    from w4a4_quantized_linear_cube_amd import dq
    return dq


def _weight(dqm, ci, co, rank, seed, spread=8):
    rng = np.random.default_rng(seed)
    rc = rng.integers(0, 256, (co, ci // 2), dtype=np.uint8)
    rs = rng.integers(127 - spread, 127, (co, ci // 32), dtype=np.uint8)
    l1, l2 = _random_factors(ci, co, rank, seed + 1)
    w = dqm.dq_import_weights(rc, rs, l1 if rank else None, l2 if rank else None)
    return w, rc, rs, l1, l2


def _x(n, ci, kind, seed):
    """(device arguments, fp64 values) of random rows."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, ci, generator=g) * torch.exp(torch.randn(ci, generator=g))
    if kind == "mx8":
        codes, scales = mx.mx_quantize(x.numpy(), "fp8")
        return ((torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV)), mx.mx_dequantize(codes, scales, "fp8"))
    x = x.to(TYPES[kind])
    return (x.to(DEV),), x.double().numpy()


def _call(dqm, w, args, a, y, stream=None):
    (dqm.dq_linear_rows8 if len(args) == 2 else dqm.dq_linear_rows)(w, *args, a, y, stream)


def _check(y, x64, rc, rs, l1, l2, parts, ytype):
    want, main, low = rows.product(x64, rc, rs, l1, l2)
    got = y.double().cpu().numpy()
    assert not np.isnan(got).any(), "unwritten outputs"
    ci, rank = x64.shape[1], l1.shape[1]
    lim = 2.0 ** -23 * ((parts * ci + 8) * main + (parts * ci + 2 * rank + 8) * low)
    lim = lim + HALF[ytype] * (np.abs(want) + lim)
    over = np.abs(got - want) / np.maximum(lim, 1e-300)
    assert over.max() <= 1.0, f"{(over > 1).sum()} outputs outside the bound, worst {over.max():.2f}x at {np.argwhere(over > 1)[:4]}"
    return np.linalg.norm(got - want) / np.linalg.norm(want)


SHAPES = [  # n, ci, co, rank
    (1, 32, 1, 0), (1, 256, 16, 1), (1, 1536, 1536, 32), (2, 96, 33, 8), (5, 416, 257, 16), (15, 128, 300, 32), (16, 2080, 1000, 40),
    (1, 5120, 13824, 32), (3, 1024, 16400, 128), (17, 1184, 515, 32), (32, 640, 1027, 64), (33, 992, 260, 0), (47, 2080, 4999, 16),
    (64, 1536, 770, 32), (65, 544, 300, 32), (130, 288, 290, 96), (8, 13824, 640, 32), (64, 13824, 129, 128),
    # every form by rows, rank and output channels: 1, up to 4, up to 16 rows; rank none or up to 32; below 8192 outputs and above
    (1, 992, 300, 0), (4, 992, 301, 0), (16, 992, 302, 0), (1, 640, 8200, 0), (4, 640, 8201, 0), (12, 640, 8202, 0),
    (1, 640, 8199, 32), (2, 640, 8200, 17), (16, 640, 8201, 32), (5, 1600, 17000, 32), (64, 3104, 10300, 32), (33, 3104, 10241, 100),
    (50, 3104, 10250, 0), (1, 20480, 96, 0), (3, 20480, 50, 32), (20, 7712, 33, 5),
    # long K without low ranks: up to 8 and up to 16 rows by 16 waves, and shared out
    (1, 16384, 70, 0), (4, 12000, 65, 0), (8, 13824, 300, 0), (16, 10240, 100, 0), (16, 13824, 96, 0), (4, 7712, 8300, 0),
    # one row with low ranks up to 48 steps, and past them; the largest rank
    (1, 6144, 40, 8), (1, 6176, 40, 8), (2, 2976, 129, 32), (2, 3136, 129, 32), (1, 640, 200, 128), (40, 9000 // 32 * 32, 513, 128),
    # 33 to 64 ranks in the form of few rows, up to 14 steps and past them, and 65
    (1, 96, 40, 33), (3, 1792, 300, 64), (16, 1056, 8200, 64), (1, 1824, 77, 48), (4, 640, 129, 64), (2, 640, 129, 65),
    (16, 992, 8200, 64), (9, 992, 100, 50), (5, 1024, 70, 8), (7, 1056, 70, 8), (16, 2176, 100, 0), (6, 2208, 8192, 0)]


@pytest.mark.parametrize("n,ci,co,rank", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "f32", "mx8"])
def test_random(dqm, n, ci, co, rank, kind):
    _say(f"rows {n} {ci}->{co} rank {rank} {kind}")
    w, rc, rs, l1, l2 = _weight(dqm, ci, co, rank, n + ci + co)
    args, x64 = _x(n, ci, kind, n)
    a = dqm.dq_rows_create(w, n)
    for ytype in ("f32", "bf16"):
        y = torch.full((n, co), float("nan"), dtype=TYPES[ytype], device=DEV)
        _call(dqm, w, args, a, y)
        rel = _check(y, x64, rc, rs, l1, l2, 3 if kind == "f32" else 1, ytype)
        assert rel <= (2e-6 if ytype == "f32" else 4e-3), rel      # (rounding errors of a sum of Ci terms in shares, taken as random)


@pytest.mark.parametrize("n,ci,co", [(1, 1536, 500), (3, 4224, 70), (16, 2080, 515), (20, 1600, 300), (64, 928, 257), (100, 352, 131)])
@pytest.mark.parametrize("kind", ["bf16", "f32", "mx8"])
def test_exact_sums(dqm, n, ci, co, kind):
    """Integers: |x| <= 8 (bf16, mx8) or up to 2^12 in 24 places (fp32, which
    needs its second part), weights multiples of 1/2 up to 12, so every partial
    sum is a multiple of 1/2 below 2^23."""
    rng = np.random.default_rng(n + ci)
    rc = rng.integers(0, 256, (co, ci // 2), dtype=np.uint8)
    rs = rng.integers(127, 129, (co, ci // 32), dtype=np.uint8)
    w = dqm.dq_import_weights(rc, rs, None, None)
    x = rng.integers(-8, 9, (n, ci)).astype(np.float32)
    if kind == "f32":
        x[:] = 0
        for i in range(n):
            x[i, rng.choice(ci, 24, replace=False)] = rng.integers(-4095, 4096, 24)
    if kind == "mx8":
        codes, scales = mx.mx_quantize(x, "fp8")
        assert np.array_equal(mx.mx_dequantize(codes, scales, "fp8"), x)
        args = (torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV))
    else:
        args = (torch.from_numpy(x).to(TYPES[kind]).to(DEV),)
    y = torch.full((n, co), float("nan"), device=DEV)
    _call(dqm, w, args, dqm.dq_rows_create(w, n), y)
    want, _, _ = rows.product(x, rc, rs, None, None)
    assert np.abs(want).max() < 2 ** 23
    assert np.array_equal(y.cpu().numpy().astype(np.float64), want)


def test_fp32_rows_keep_all_their_bits(dqm):
    """One 24-bit value per row against one weight: the product is exact to the last bit."""
    ci, co = 256, 48
    rng = np.random.default_rng(3)
    rc, rs = np.full((co, ci // 2), 0x22, np.uint8), rng.integers(100, 150, (co, ci // 32), dtype=np.uint8)
    w = dqm.dq_import_weights(rc, rs, None, None)
    n = 40
    x = np.zeros((n, ci), np.float32)
    at = rng.integers(0, ci, n)
    x[np.arange(n), at] = (rng.integers(2 ** 23, 2 ** 24, n) * np.where(rng.random(n) < 0.5, -1, 1)).astype(np.float32)
    y = torch.empty(n, co, device=DEV)
    dqm.dq_linear_rows(w, torch.from_numpy(x).to(DEV), dqm.dq_rows_create(w, n), y)
    want, _, _ = rows.product(x, rc, rs, None, None)
    assert np.array_equal(y.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("code", [0, 1, 3, 64, 190, 250, 252])
def test_extreme_weight_scales(dqm, code):
    """Scales 2^-127 to 2^125 against rows that bring the products back to the
    size of 1: one nonzero channel a row, so each output is one exact product
    (weights below 2^-126 are subnormal in bf16, and must not vanish)."""
    ci, co, n = 160, 64, 5
    rng = np.random.default_rng(code)
    rc, rs = rng.integers(0, 256, (co, ci // 2), dtype=np.uint8), np.full((co, ci // 32), code, np.uint8)
    w = dqm.dq_import_weights(rc, rs, None, None)
    x = np.zeros((n, ci), np.float32)
    at = rng.integers(0, ci, n)
    x[np.arange(n), at] = np.ldexp(rng.integers(1, 8, n).astype(np.float32), 127 - code if code > 10 else 120)
    want, _, _ = rows.product(x, rc, rs, None, None)
    a = dqm.dq_rows_create(w, 40)
    for t in (torch.float32, torch.bfloat16):
        for m in (n, 8 * n):                                  # a form of its own for many rows
            y = torch.empty(m, co, device=DEV)
            dqm.dq_linear_rows(w, torch.from_numpy(np.tile(x, (m // n, 1))).to(t).to(DEV), a, y)
            assert np.array_equal(y.cpu().numpy().astype(np.float64), np.tile(want, (m // n, 1)))


def test_two_workspaces_on_two_streams(dqm):
    """Calls that overlap on one GPU, each with its own workspace."""
    w, rc, rs, l1, l2 = _weight(dqm, 4096, 640, 32, 31)
    cases = []
    for i, n in enumerate((3, 24, 64)):
        args, x64 = _x(n, 4096, "bf16", i)
        cases.append((torch.cuda.Stream(), args, x64, dqm.dq_rows_create(w, n), torch.full((n, 640), float("nan"), device=DEV)))
    torch.cuda.synchronize()
    for _ in range(20):
        for stream, args, _, a, y in cases:
            dqm.dq_linear_rows(w, *args, a, y, stream)
    torch.cuda.synchronize()
    for _, _, x64, _, y in cases:
        _check(y, x64, rc, rs, l1, l2, 1, "f32")


def test_low_rank_alone(dqm):
    """A zero residual: y = (x L1) L2 exactly on integers, every rank place used."""
    ci, co, rank, n = 160, 77, 37, 18
    rng = np.random.default_rng(9)
    bits = lambda v: mx.f32_to_bf16_bits(v.astype(np.float32))
    l1, l2 = bits(rng.integers(-2, 3, (ci, rank))), bits(rng.integers(-2, 3, (rank, co)))
    w = dqm.dq_import_weights(np.zeros((co, ci // 2), np.uint8), np.zeros((co, ci // 32), np.uint8), l1, l2)
    x = rng.integers(-4, 5, (n, ci)).astype(np.float32)
    y = torch.empty(n, co, device=DEV)
    a = dqm.dq_rows_create(w, n)
    for t in (torch.bfloat16, torch.float32):
        y.fill_(float("nan"))
        dqm.dq_linear_rows(w, torch.from_numpy(x).to(t).to(DEV), a, y)
        want, _, _ = rows.product(x, np.zeros((co, ci // 2), np.uint8), np.zeros((co, ci // 32), np.uint8), l1, l2)
        assert np.array_equal(y.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_strided_rows_and_untouched_neighbours(dqm, kind):
    n, ci, co = 11, 352, 123
    w, rc, rs, l1, l2 = _weight(dqm, ci, co, 16, 77)
    wide = torch.randn(n, ci + 48, generator=torch.Generator().manual_seed(5)).to(TYPES[kind]).to(DEV)
    x = wide[:, 16:16 + ci]
    out = torch.full((n + 2, co + 9), 3.0, device=DEV)
    dqm.dq_linear_rows(w, x, dqm.dq_rows_create(w, 16), out[1:n + 1, 4:4 + co])
    _check(out[1:n + 1, 4:4 + co], x.double().cpu().numpy(), rc, rs, l1, l2, 3 if kind == "f32" else 1, "f32")
    out[1:n + 1, 4:4 + co] = 3.0
    assert (out == 3.0).all()


def test_prepared_and_imported_weights_agree(dqm):
    """A prepared weight exported and imported again: the same export, and the same products bit for bit; an imported weight serves dq_linear too."""
    from w4a4_quantized_linear_cube_amd import synth
    ci, co, rank = 224, 300, 16
    wt = synth.make_weight(ci, co, seed=5, dtype="bf16")
    l1, l2 = _random_factors(ci, co, rank, 6)
    p = dqm.dq_prepare_weights_lowrank(wt, l1, l2)
    e = dqm.dq_weights_export(p)
    q = dqm.dq_import_weights(e["rcodes"], e["rscales"], e["l1"], e["l2"])
    f = dqm.dq_weights_export(q)
    for k in ("l1", "l2", "rcodes", "rscales"):
        assert np.array_equal(e[k], f[k]), k
    assert np.array_equal(f["r"].astype(np.float64), rows.weight_values(e["rcodes"], e["rscales"]))
    x = torch.randn(6, ci, generator=torch.Generator().manual_seed(1)).to(DEV)
    y = [torch.empty(6, co, device=DEV) for _ in range(4)]
    a = dqm.dq_rows_create(p, 6)
    dqm.dq_linear_rows(p, x, a, y[0])
    dqm.dq_linear_rows(q, x, a, y[1])                        # (the workspace serves every weight of these sizes)
    geom = (1, 2, 3, 1, 2, 2)
    for w, out in ((p, y[2]), (q, y[3])):
        dqm.dq_linear(w, x, dqm.dq_qact_create(w, geom), out)
    assert torch.equal(y[0], y[1]) and torch.equal(y[2], y[3])


def test_more_rows_then_fewer(dqm):
    """A workspace's older, longer contents (other row kinds too) do not reach a later call."""
    ci, co = 416, 200
    w, rc, rs, l1, l2 = _weight(dqm, ci, co, 32, 15)
    a = dqm.dq_rows_create(w, 100)
    nan = torch.full((100, ci), float("nan"), device=DEV)
    junk = torch.empty(100, co, device=DEV)
    for n, kind in ((100, "f32"), (3, "bf16"), (40, "mx8"), (1, "f32"), (70, "bf16")):
        dqm.dq_linear_rows(w, nan, a, junk)
        assert torch.isnan(junk).all()
        args, x64 = _x(n, ci, kind, n)
        y = torch.full((n, co), float("nan"), device=DEV)
        _call(dqm, w, args, a, y)
        _check(y, x64, rc, rs, l1, l2, 3, "f32")


def test_nan_and_infinite_values_stay_in_their_rows(dqm):
    ci, co, n = 256, 100, 20
    rng = np.random.default_rng(2)
    rc = (rng.integers(1, 8, (co, ci // 2)) | rng.integers(1, 8, (co, ci // 2)) << 4).astype(np.uint8)     # no zero weights, all positive
    rs = np.full((co, ci // 32), 127, np.uint8)
    w = dqm.dq_import_weights(rc, rs, None, None)
    a = dqm.dq_rows_create(w, n)
    x = torch.randn(n, ci, generator=torch.Generator().manual_seed(1))
    x[3, 100], x[7, 5], x[19, 255] = float("nan"), float("inf"), float("-inf")
    for t in (torch.float32, torch.bfloat16):
        y = torch.empty(n, co, device=DEV)
        dqm.dq_linear_rows(w, x.to(t).to(DEV), a, y)
        assert torch.isnan(y[3]).all() and (y[7] == float("inf")).all() and (y[19] == float("-inf")).all()
        rest = [i for i in range(n) if i not in (3, 7, 19)]
        assert torch.isfinite(y[rest]).all()
    codes = torch.full((n, ci), 0x38, dtype=torch.uint8, device=DEV)
    scales = torch.full((n, ci // 32), 127, dtype=torch.uint8, device=DEV)
    codes[2, 9], scales[5, 7] = 0x7F, 255
    y = torch.empty(n, co, device=DEV)
    dqm.dq_linear_rows8(w, codes, scales, a, y)
    nan = torch.isnan(y)
    assert nan[2].all() and nan[5].all() and nan.sum() == 2 * co


def test_twice_the_same_on_streams_and_in_graphs(dqm):
    """Repeated calls agree bit for bit; so do a side stream, and a captured
    norm and two products replayed on new inputs with eager work between."""
    n, c = 4, 1536
    wq, *_ = _weight(dqm, c, c, 32, 91)
    wk, *_ = _weight(dqm, c, 2 * c - 40, 32, 92)
    aq, ak = dqm.dq_rows_create(wq, n), dqm.dq_rows_create(wk, n)
    x, r = (torch.empty(n, c, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    codes, scales = torch.empty(n, c, dtype=torch.uint8, device=DEV), torch.empty(n, c // 32, dtype=torch.uint8, device=DEV)
    h = torch.empty_like(x)
    out = [torch.empty(n, co, dtype=torch.bfloat16, device=DEV) for co in (c, 2 * c - 40)]

    def step(stream=None):
        dqm.dq_rmsnorm8(x, None, 1e-6, codes, scales, residual=r, h=h, stream=stream)
        dqm.dq_linear_rows8(wq, codes, scales, aq, out[0], stream)
        dqm.dq_linear_rows8(wk, codes, scales, ak, out[1], stream)

    def fill(i):
        g = torch.Generator(device=DEV).manual_seed(i)
        x.copy_(torch.randn(n, c, generator=g, device=DEV))
        r.copy_(torch.randn(n, c, generator=g, device=DEV))

    def eager(i):
        fill(i)
        step()
        torch.cuda.synchronize()
        return [t.clone() for t in (codes, scales, h, *out)]

    want = [eager(i) for i in range(4)]
    for i, e in enumerate(want):
        assert all(torch.equal(p, q) for p, q in zip(e, eager(i)))
    side = torch.cuda.Stream()
    fill(2)
    side.wait_stream(torch.cuda.current_stream())
    for t in out:
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want[2], (codes, scales, h, *out)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in (1, 3, 0, 1):
        fill(i)
        for t in out:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want[i], (codes, scales, h, *out))), i
        eager(2)                                              # eager calls through the same workspaces between replays


def test_a_run_of_blocks(dqm):
    """norm -> two products -> norm of their sum with the stream, three times
    over, as a decoding loop would; each step against the oracle from the
    GPU's own stream."""
    n, c = 3, 512
    ws = [_weight(dqm, c, c, 16, 200 + i, spread=10) for i in range(3)]
    a = dqm.dq_rows_create(ws[0][0], n)
    g = torch.Generator().manual_seed(8)
    h = torch.randn(n, c, generator=g).to(torch.bfloat16).to(DEV)
    y = torch.randn(n, c, generator=g).to(torch.bfloat16).to(DEV)
    codes, scales = torch.empty(n, c, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(n, c // 32, dtype=torch.uint8, device=DEV)
    gain = (1 + 0.1 * torch.randn(c, generator=g)).to(torch.bfloat16).to(DEV)
    for w, rc, rs, l1, l2 in ws:
        before, added = h.float().cpu().numpy(), y.float().cpu().numpy()
        dqm.dq_rmsnorm8(y, gain, 1e-6, codes, scales, residual=h, h=h)
        want = rows.rms_norm8(added, before, gain.float().cpu().numpy(), 1e-6, "bf16")
        assert np.array_equal(h.float().cpu().numpy(), want["h"])
        assert np.array_equal(codes.view(torch.uint8).cpu().numpy(), want["codes"])
        dqm.dq_linear_rows8(w, codes, scales, a, y)
        _check(y, mx.mx_dequantize(want["codes"], want["scales"], "fp8"), rc, rs, l1, l2, 1, "bf16")


def test_refused_on_device(dqm):
    w, *_ = _weight(dqm, 64, 40, 8, 1)
    a = dqm.dq_rows_create(w, 4)
    x, y = torch.zeros(5, 64, device=DEV), torch.full((5, 40), 2.0, device=DEV)
    f = dqm.dq_linear_rows
    with pytest.raises(dqm.DQError, match="max_rows"):
        f(w, x, a, y)
    with pytest.raises(dqm.DQError, match="shape"):
        f(w, x[:4], a, y)
    with pytest.raises(dqm.DQError, match="aligned"):
        f(w, torch.zeros(4, 65, device=DEV)[:, 1:], a, y[:4])
    with pytest.raises(dqm.DQError, match="dtype"):
        f(w, x[:4], a, y[:4].half())
    other, *_ = _weight(dqm, 64, 41, 8, 1)
    with pytest.raises(dqm.DQError, match="different weight"):
        f(other, x[:4], a, torch.zeros(4, 41, device=DEV))
    for bad in (0, 4097):
        with pytest.raises(dqm.DQError, match="max_rows"):
            dqm.dq_rows_create(w, bad)
    six = dqm.dq_prepare_weights_w6(torch.zeros(40, 64), None, None)
    with pytest.raises(dqm.DQError, match="6-bit"):
        dqm.dq_rows_create(six, 4)
    with pytest.raises(dqm.DQError, match="overlaps"):
        both = torch.zeros(4, 104, device=DEV)
        f(w, both[:, :64], a, both[:, 60:100])
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8, device=DEV), torch.zeros(4, 2, dtype=torch.uint8, device=DEV)
    with pytest.raises(dqm.DQError, match="shape"):
        dqm.dq_linear_rows8(w, codes, scales[:, :1], a, y[:4])
    with pytest.raises(dqm.DQError, match="cuda:0"):
        dqm.dq_linear_rows8(w, codes, scales.cpu(), a, y[:4])
    f(w, x[:0], a, y[:0])                                     # no rows: nothing happens
    torch.cuda.synchronize()
    assert (y == 2.0).all()


@pytest.mark.parametrize("rank", [0, 5, 32, 37, 64, 128])
@pytest.mark.parametrize("n", [1, 3, 20])
def test_infinite_channels_with_low_ranks(dqm, n, rank):
    """Positive weights and factors: a row with an infinite channel is infinite,
    also where the rank does not fill its padded width; a NaN stays in its row."""
    ci, co = 288, 140
    rng = np.random.default_rng(rank)
    rc = (rng.integers(1, 8, (co, ci // 2)) | rng.integers(1, 8, (co, ci // 2)) << 4).astype(np.uint8)
    rs = np.full((co, ci // 32), 127, np.uint8)
    bits = lambda v: mx.f32_to_bf16_bits(v.astype(np.float32))
    l1, l2 = (bits(rng.integers(1, 4, s)) for s in ((ci, rank), (rank, co)))
    w = dqm.dq_import_weights(rc, rs, l1 if rank else None, l2 if rank else None)
    a = dqm.dq_rows_create(w, n)
    x = torch.ones(n, ci)
    x[0, 287] = float("-inf")
    if n > 2:
        x[2, 3] = float("nan")
    for t in (torch.float32, torch.bfloat16):
        y = torch.zeros(n, co, device=DEV)
        dqm.dq_linear_rows(w, x.to(t).to(DEV), a, y)
        assert (y[0] == float("-inf")).all()
        assert n == 1 or torch.isnan(y[2]).all() and torch.isfinite(y[[i for i in range(1, n) if i != 2]]).all()


@pytest.mark.parametrize("kind", ["f32", "mx8"])
@pytest.mark.parametrize("n", [2, 24])
def test_tiny_values(dqm, n, kind):
    """Values of multiples of 2^-133 (subnormal parts in bf16) against scales of
    2^120, one a row.  An fp32 value here has up to 23 bits and a weight 2, so
    their product has up to 25 and takes one rounding (the first two parts'
    products have 10 bits each and sum exactly; only the third addition
    rounds, by 2^-23 of the sum where it truncates); an MX-FP8 product is exact."""
    ci, co = 96, 50
    rng = np.random.default_rng(n)
    rc, rs = rng.integers(0, 256, (co, ci // 2), dtype=np.uint8), np.full((co, ci // 32), 247, np.uint8)
    w = dqm.dq_import_weights(rc, rs, None, None)
    a, y = dqm.dq_rows_create(w, n), torch.empty(n, co, device=DEV)
    at = rng.integers(0, ci, n)
    if kind == "f32":
        x = np.zeros((n, ci), np.float32)
        x[np.arange(n), at] = np.ldexp(rng.integers(2 ** 19, 2 ** 22, n).astype(np.float32) * 2 + 1, -133)
        args = (torch.from_numpy(x).to(DEV),)
    else:
        codes, scales = np.zeros((n, ci), np.uint8), np.full((n, ci // 32), 3, np.uint8)       # 2^-124, least code 2^-9
        codes[np.arange(n), at] = rng.integers(1, 0x7F, n)
        args, x = (torch.from_numpy(codes).to(DEV), torch.from_numpy(scales).to(DEV)), mx.mx_dequantize(codes, scales, "fp8")
    _call(dqm, w, args, a, y)
    want, _, _ = rows.product(x, rc, rs, None, None)
    assert (np.abs(y.cpu().numpy() - want) <= (2.0 ** -23 if kind == "f32" else 0.0) * np.abs(want)).all()


@pytest.mark.parametrize("n,ci,co,rank", [(1, 8320, 200, 32), (24, 1024, 130, 40), (64, 3104, 10250, 32)])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_shared_tiles_in_graphs(dqm, n, ci, co, rank, kind):
    """Products whose tiles several workgroups share, captured and replayed on new rows, with eager calls through the same workspace between."""
    w, *_ = _weight(dqm, ci, co, rank, ci)
    a = dqm.dq_rows_create(w, n)
    many = [_x(n, ci, kind, 50 + i)[0][0] for i in range(3)]
    x, y = torch.empty_like(many[0]), torch.empty(n, co, device=DEV)

    def eager(i):
        x.copy_(many[i])
        dqm.dq_linear_rows(w, x, a, y)
        return y.clone()

    want = [eager(i) for i in range(3)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dqm.dq_linear_rows(w, x, a, y)
        dqm.dq_linear_rows(w, x, a, y)                        # (one after the other: the workspace is ready for the next)
    for i in (1, 0, 2, 1):
        x.copy_(many[i])
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i]), i
        assert torch.equal(eager(2), want[2])


def test_host_threads(dqm):
    """Calls from several threads on one weight, each with its own workspace and stream (given as its raw value)."""
    import threading
    n, ci, co = 20, 1536, 300
    w, rc, rs, l1, l2 = _weight(dqm, ci, co, 32, 3)
    args, x64 = _x(n, ci, "mx8", 4)
    jobs = [(dqm.dq_rows_create(w, n), torch.full((n, co), float("nan"), device=DEV), torch.cuda.Stream()) for _ in range(4)]
    torch.cuda.synchronize()
    errors = []

    def run(a, y, stream):
        try:
            for _ in range(50):
                dqm.dq_linear_rows8(w, *args, a, y, stream.cuda_stream)
            with pytest.raises(dqm.DQError, match="max_rows"):
                dqm.dq_linear_rows8(w, *(torch.cat((t, t)) for t in args), a, torch.cat((y, y)))
        except BaseException as e:
            errors.append(e)

    threads = [threading.Thread(target=run, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for _, y, _ in jobs:
        _check(y, x64, rc, rs, l1, l2, 1, "f32")


@pytest.mark.parametrize("n,ci,co,rank", [(4096, 160, 130, 32), (4095, 96, 70, 0), (2, 65536, 40, 32), (16, 65536, 33, 0), (33, 65536, 20, 5)])
@pytest.mark.parametrize("kind", ["bf16", "f32", "mx8"])
def test_largest_sizes(dqm, n, ci, co, rank, kind):
    """The most rows a workspace takes, and the longest K."""
    _say(f"largest {n} {ci}->{co} rank {rank} {kind}")
    w, rc, rs, l1, l2 = _weight(dqm, ci, co, rank, 5)
    args, x64 = _x(n, ci, kind, 6)
    y = torch.full((n + 1, co), float("nan"), device=DEV)
    _call(dqm, w, args, dqm.dq_rows_create(w, n), y[:n])
    _check(y[:n], x64, rc, rs, l1, l2, 3 if kind == "f32" else 1, "f32")
    assert torch.isnan(y[n]).all()


def test_longer_rows_are_refused(dqm):
    w, *_ = _weight(dqm, 65568, 20, 0, 5)
    with pytest.raises(dqm.DQError, match="65536"):
        dqm.dq_rows_create(w, 1)
