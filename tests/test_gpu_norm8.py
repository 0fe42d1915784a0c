"""dq_rmsnorm8 on the GPU against the oracle: h, codes and scale codes bit for
bit, plain values bit for bit (their one rounding to the stream's type is
defined by the format)."""
import numpy as np
import pytest
import torch

from oracle import mx, rows
from parity_util import DEV, _say

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dqm(lib):
    from w4a4_quantized_linear_cube_amd import dq
    return dq


def _stream_rows(n, c, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, c, generator=g) * torch.exp(spread * torch.randn(c, generator=g))
    x[:, torch.randint(0, c, (max(1, c // 256),), generator=g)] *= 40.0
    return x.to(TYPES[dtype])


def _f32(t):
    return t.detach().float().cpu().numpy()


def _bits(t):
    t = t.detach().cpu()
    return t.view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2 else torch.int32).numpy()


def _outputs(n, c, dtype):
    return (torch.full((n, c), 0x55, dtype=torch.uint8, device=DEV), torch.full((n, c // 32), 0x55, dtype=torch.uint8, device=DEV),
            torch.full((n, c), float("nan"), dtype=TYPES[dtype], device=DEV),
            torch.full((n, c), float("nan"), dtype=TYPES[dtype], device=DEV))


def _compare(want, codes, scales, h=None, y=None, dtype="bf16"):
    assert np.array_equal(_bits(scales), want["scales"]), "scale codes"
    assert np.array_equal(_bits(codes), want["codes"]), "codes"
    if h is not None:
        assert np.array_equal(_f32(h).view(np.uint32), want["h"].view(np.uint32)), "h"
    if y is not None:
        assert np.array_equal(_f32(y).view(np.uint32), rows.to_stream(want["v"], dtype).view(np.uint32)), "plain values"


# Every number of 8-channel chunks a thread can hold, at both ends of each
# width (threads to a row), rows that do not fill a workgroup, one row, many
# rows: those of up to 3 2^20 elements take one form, larger ones another.
SHAPES = [(1, 32), (3, 32), (5, 64), (7, 512), (4, 544), (9, 1024), (2, 1536), (6, 2048), (1, 2080), (3, 4096), (2, 5120),
          (2, 6176), (3, 8192), (1, 8224), (2, 13824), (1, 16384), (2, 24608), (1, 32768), (1031, 96), (517, 1536), (130, 5120),
          (32801, 96), (6200, 512), (3111, 1024), (2051, 1536), (1541, 2048), (1513, 2080), (771, 4096), (615, 5120), (387, 8192),
          (383, 8224), (229, 13824), (193, 16384), (129, 24608), (97, 32768)]


@pytest.mark.parametrize("n,c", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sizes(dqm, n, c, dtype):
    _say(f"norm8 {n}x{c} {dtype}")
    x, r = _stream_rows(n, c, dtype, c + n), 2 * _stream_rows(n, c, dtype, c + n + 1)
    gain = 1 + 0.3 * torch.randn(c, generator=torch.Generator().manual_seed(3))
    codes, scales, h, y = _outputs(n, c, dtype)
    dqm.dq_rmsnorm8(x.to(DEV), gain.to(DEV), 1e-6, codes, scales, residual=r.to(DEV), h=h, y=y)
    want = rows.rms_norm8(_f32(x), _f32(r), gain.numpy(), 1e-6, dtype)
    _compare(want, codes, scales, h, y, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("residual,gain,outs", [(False, None, "codes"), (True, "bf16", "codes"), (False, "f32", "y"),
                                                (True, "f32", "y"), (True, None, "all")])
def test_forms(dqm, dtype, group, residual, gain, outs):
    n, c = 37, 1600
    x = _stream_rows(n, c, dtype, 11)
    r = _stream_rows(n, c, dtype, 12) if residual else None
    g = None if gain is None else torch.randn(c, generator=torch.Generator().manual_seed(13)).to(TYPES[gain])
    codes, scales, h, y = _outputs(n, c, dtype)
    dqm.dq_rmsnorm8(x.to(DEV), None if g is None else g.to(DEV), 1e-5, *((None, None) if outs == "y" else (codes, scales)),
                    residual=None if r is None else r.to(DEV), h=h if residual and outs != "codes" else None,
                    y=None if outs == "codes" else y, group=group)
    want = rows.rms_norm8(_f32(x), None if r is None else _f32(r), None if g is None else _f32(g), 1e-5, dtype, group)
    if outs == "y":
        assert (codes == 0x55).all() and (scales == 0x55).all()
        assert np.array_equal(_f32(y).view(np.uint32), rows.to_stream(want["v"], dtype).view(np.uint32))
    else:
        _compare(want, codes, scales, h if residual and outs == "all" else None, y if outs == "all" else None, dtype)


def test_float8_tensors_and_strides(dqm):
    """Views into wider buffers: rows 8 elements (16 bytes) off and apart; what lies between the rows stays."""
    n, c = 21, 416
    buf = _stream_rows(n, c + 40, "bf16", 21).to(DEV)
    res = _stream_rows(n, c + 8, "bf16", 22).to(DEV)
    out = torch.full((n, 2 * c + 16), 7.0, dtype=torch.bfloat16, device=DEV)
    x, r, h, y = buf[:, 8:8 + c], res[:, :c], out[:, :c], out[:, c + 8:2 * c + 8]
    codes = torch.empty(n, c, dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(n, c // 32, dtype=torch.float8_e8m0fnu, device=DEV)
    dqm.dq_rmsnorm8(x, None, 1e-6, codes, scales, residual=r, h=h, y=y)
    want = rows.rms_norm8(_f32(x), _f32(r), None, 1e-6, "bf16")
    _compare(want, codes, scales, h, y)
    assert (out[:, c:c + 8] == 7).all() and (out[:, 2 * c + 8:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(dqm, dtype):
    """h over the residual, y over x: what a serving loop does."""
    n, c = 19, 5120
    x, r = _stream_rows(n, c, dtype, 31), _stream_rows(n, c, dtype, 32)
    want = rows.rms_norm8(_f32(x), _f32(r), None, 1e-6, dtype)
    codes, scales, _, _ = _outputs(n, c, dtype)
    xd, rd = x.to(DEV), r.to(DEV)
    dqm.dq_rmsnorm8(xd, None, 1e-6, codes, scales, residual=rd, h=rd, y=xd)
    _compare(want, codes, scales, rd, xd, dtype)


def test_zero_rows_and_no_rows(dqm):
    c = 256
    x = torch.zeros(4, c, device=DEV)
    x[1] = -0.0
    x[3, 5] = 2.0 ** -140                                     # a subnormal alone
    codes, scales, _, y = _outputs(4, c, "f32")
    dqm.dq_rmsnorm8(x, None, 1e-12, codes, scales, y=y)
    _compare(rows.rms_norm8(_f32(x), None, None, 1e-12, "f32"), codes, scales, None, y, "f32")
    assert (scales[0] == 0).all() and (codes[0] == 0).all() and (codes[1] == 0x80).all()
    codes[:] = 9
    dqm.dq_rmsnorm8(x[:0], None, 1e-12, codes[:0], scales[:0])
    assert (codes == 9).all()


def test_extreme_magnitudes(dqm):
    """Squares that leave fp32's range: the sum is kept in fp64."""
    g = torch.Generator().manual_seed(41)
    x = torch.randn(6, 128, generator=g) * torch.tensor([1e30, 1e37, 1e-25, 1e-38, 1.0, 3e4])[:, None]
    codes, scales, _, y = _outputs(6, 128, "f32")
    dqm.dq_rmsnorm8(x.to(DEV), None, 1e-50, codes, scales, y=y)
    want = rows.rms_norm8(x.numpy(), None, None, 1e-50, "f32")
    _compare(want, codes, scales, None, y, "f32")
    assert np.isfinite(want["v"]).all()


def test_group_maxima_beside_the_borders(dqm):
    """Gains that put a group's maximum on 448 2^e and one step to either side,
    and elements on midpoints of E4M3: rows of +-1 have f = 1 exactly with
    a vanishing eps, so v is the gain itself."""
    c = 1024
    g = torch.Generator().manual_seed(51)
    x = torch.where(torch.rand(3, c, generator=g) < 0.5, -1.0, 1.0)
    gain = torch.empty(c)
    mids = np.array([(mx.fp8_decode_magnitude(i) + mx.fp8_decode_magnitude(i + 1)) / 2 for i in range(126)], np.float32)
    for k in range(c // 32):
        top = np.float32(448.0 * 2.0 ** (k % 7 - 3))
        top = [top, np.nextafter(top, np.float32(0)), np.nextafter(top, np.float32(np.inf))][k % 3]
        vals = mids[(np.arange(31) * 4 + k) % 126] * np.float32(2.0 ** (k % 7 - 3))
        gain[32 * k:32 * k + 32] = torch.from_numpy(np.concatenate([[top], vals]).astype(np.float32))
    codes, scales, _, _ = _outputs(3, c, "f32")
    dqm.dq_rmsnorm8(x.to(DEV), gain.to(DEV), 1e-60, codes, scales)
    want = rows.rms_norm8(x.numpy(), None, gain.numpy(), 1e-60, "f32")
    assert np.array_equal(np.abs(want["v"][0]), gain.numpy())
    _compare(want, codes, scales)


def test_nan_and_infinite_rows(dqm):
    """A NaN spoils its row, an infinity makes its row zeros with a NaN in its
    own place, an overflowing gain its own element; other rows are untouched,
    and a NaN takes no part in its group's scale."""
    n, c = 5, 128
    x = _stream_rows(n, c, "f32", 61, 0.2)
    gain = torch.ones(c)
    gain[40] = 3e38
    x[1, 7], x[2, 33], x[4, 40] = float("nan"), float("-inf"), 1e3
    codes, scales, _, y = _outputs(n, c, "f32")
    dqm.dq_rmsnorm8(x.to(DEV), gain.to(DEV), 1e-6, codes, scales, y=y)
    with np.errstate(all="ignore"):
        _, v = rows.rms_norm(x.numpy(), None, gain.numpy(), 1e-6, "f32")
    got = y.cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(v))
    live = ~np.isnan(v)
    assert np.array_equal(got[live], v[live])
    finite = np.isfinite(v)
    assert not finite[1].any() and (~finite[2]).sum() == 1 and not finite[4, 40]
    wc, ws = mx.mx_quantize(np.where(finite, v, 0).astype(np.float32), "fp8")
    got = codes.cpu().numpy()
    assert np.array_equal(scales.cpu().numpy(), ws)
    assert np.array_equal(got[finite], wc[finite])
    assert ((got[~finite] & 0x7F) == 0x7F).all()


def test_other_stream_and_graph(dqm):
    """A side stream's order, and a captured call replayed on new inputs."""
    n, c = 64, 1536
    codes, scales, h, y = _outputs(n, c, "bf16")
    x, r = torch.empty(n, c, dtype=torch.bfloat16, device=DEV), torch.empty(n, c, dtype=torch.bfloat16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x.copy_(_stream_rows(n, c, "bf16", 71))
        r.copy_(_stream_rows(n, c, "bf16", 72))
        dqm.dq_rmsnorm8(x, None, 1e-6, codes, scales, residual=r, h=h, y=y)
    side.synchronize()
    _compare(rows.rms_norm8(_f32(x), _f32(r), None, 1e-6, "bf16"), codes, scales, h, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dqm.dq_rmsnorm8(x, None, 1e-6, codes, scales, residual=r, h=h, y=y)
    for i in range(3):
        x.copy_(_stream_rows(n, c, "bf16", 80 + i))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _compare(rows.rms_norm8(_f32(x), _f32(r), None, 1e-6, "bf16"), codes, scales, h, y)
        (x.float() @ x.float().t()).sum().item()                # eager work between replays


def test_refused_on_device(dqm):
    x = torch.zeros(4, 64, device=DEV)
    codes, scales, h, y = _outputs(4, 64, "f32")
    with pytest.raises(dqm.DQError, match="shape"):
        dqm.dq_rmsnorm8(x, torch.ones(32, device=DEV), 1e-6, codes, scales)
    with pytest.raises(dqm.DQError, match="dtype"):
        dqm.dq_rmsnorm8(x, None, 1e-6, codes, scales, residual=x.bfloat16())
    with pytest.raises(dqm.DQError, match="aligned"):
        dqm.dq_rmsnorm8(torch.zeros(4, 65, device=DEV)[:, 1:], None, 1e-6, codes, scales)
    with pytest.raises(dqm.DQError, match="cuda:0"):
        dqm.dq_rmsnorm8(x, None, 1e-6, codes.cpu(), scales)
    with pytest.raises(dqm.DQError, match="both codes"):
        dqm.dq_rmsnorm8(x, None, 1e-6, codes)
    with pytest.raises(dqm.DQError, match="no output"):
        dqm.dq_rmsnorm8(x, None, 1e-6)
    with pytest.raises(dqm.DQError, match="without a residual"):
        dqm.dq_rmsnorm8(x, None, 1e-6, codes, scales, h=h)
    with pytest.raises(dqm.DQError, match="overlap"):
        buf = torch.zeros(5, 64, device=DEV)
        dqm.dq_rmsnorm8(buf[:4], None, 1e-6, codes, scales, y=buf[1:])


def test_more_rows_than_one_launch_takes(dqm):
    """2^26 rows and a few, of 32 channels: offsets past 32 bits, and more threads than a launch may have."""
    _say("norm of 2^26 + 700 rows")
    period, n, c = 1 << 14, (1 << 26) + 700, 32
    base = torch.randn(period, c, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    few = [torch.empty(period, k, dtype=torch.uint8, device=DEV) for k in (c, 1)]
    dqm.dq_rmsnorm8(base, None, 1e-6, *few)
    x = base.repeat(n // period + 1, 1)[:n]
    codes, scales = (torch.full((n + 1, k), 0xA5, dtype=torch.uint8, device=DEV) for k in (c, 1))
    dqm.dq_rmsnorm8(x, None, 1e-6, codes[:n], scales[:n])
    for got, want in zip((codes, scales), few):
        whole = n // period * period
        assert (got[:whole].view(-1, period, got.shape[1]) == want).all()
        assert torch.equal(got[whole:n], want[:n - whole])
        assert (got[n:] == 0xA5).all()


@pytest.mark.parametrize("n", [1, 7, 33, 1030])
@pytest.mark.parametrize("c,group", [(32, 32), (64, 32), (64, 64), (96, 32), (128, 64), (160, 32), (192, 64), (256, 32), (288, 32), (512, 64), (544, 32)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_short_rows(dqm, n, c, group, dtype):
    """Several rows to a wave: each with its own sum and scales, none past the last touched."""
    x, r = _stream_rows(n, c, dtype, c + n), _stream_rows(n, c, dtype, c + n + 1)
    x[n // 2] = 0.0 if n > 1 else x[0]
    codes, scales, h, y = _outputs(n + 3, c, dtype)
    before = [t[n:].clone() for t in (codes, scales, h, y)]
    dqm.dq_rmsnorm8(x.to(DEV), None, 1e-5, codes[:n], scales[:n], residual=r.to(DEV), h=h[:n], y=y[:n], group=group)
    want = rows.rms_norm8(_f32(x), _f32(r), None, 1e-5, dtype, group)
    _compare(want, codes[:n], scales[:n], h[:n], y[:n], dtype)
    for t, b in zip((codes, scales, h, y), before):
        assert torch.equal(t[n:].view(torch.uint8), b.view(torch.uint8))


def test_many_short_rows(dqm):
    """Enough rows that the outputs bypass the caches, by a period of rows whose own codes are known."""
    for c, dtype in ((64, "bf16"), (128, "f32"), (448, "bf16")):
        period, n = 1000, (4 << 20) // c + 77
        base = _stream_rows(period, c, dtype, c)
        want = rows.rms_norm8(_f32(base), None, None, 1e-6, dtype)
        x = base.repeat(n // period + 1, 1)[:n].to(DEV)
        codes, scales, _, _ = _outputs(n, c, dtype)
        dqm.dq_rmsnorm8(x, None, 1e-6, codes, scales)
        for got, part in ((codes, want["codes"]), (scales, want["scales"])):
            full = torch.from_numpy(part).repeat(n // period + 1, 1)[:n]
            assert torch.equal(got.view(torch.uint8).cpu(), full)
