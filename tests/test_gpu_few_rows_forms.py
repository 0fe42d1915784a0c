"""Forms of the few-row kernels that take sizes of their own to reach: norms of
more rows than one launch takes, the widest rows' third chunk, and the direct
product with 33 to 64 low ranks and many output channels."""
import pytest
import torch

from oracle import rows
from parity_util import DEV, _say
from test_gpu_norm8 import _compare, _f32, _outputs, _stream_rows
from test_gpu_rows import TYPES, _call, _check, _weight, _x

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dqm(lib):
    from w4a4_quantized_linear_cube_amd import dq
    return dq


# A launch takes 2^31 threads: of 8 threads to a row of 32 channels 2^28 rows,
# of 64 threads to one of 288 channels 2^25.
@pytest.mark.parametrize("n,c", [((1 << 28) + 700, 32), ((1 << 25) + 700, 288)])
def test_norm_by_several_launches(dqm, n, c):
    """The second launch's rows begin where the first one's end, past 2^32 elements; the row behind the last stays."""
    _say(f"norm {n}x{c}, two launches")
    period = 1 << 14
    base = _stream_rows(period, c, "bf16", c)
    want = rows.rms_norm8(_f32(base), None, None, 1e-6, "bf16")
    x = base.to(DEV).repeat(n // period + 1, 1)[:n]
    codes, scales = (torch.full((n + 1, k), 0xA5, dtype=torch.uint8, device=DEV) for k in (c, c // 32))
    dqm.dq_rmsnorm8(x, None, 1e-6, codes[:n], scales[:n])
    for got, part in ((codes, want["codes"]), (scales, want["scales"])):
        part = torch.from_numpy(part).to(DEV)
        for at in range(0, n, 64 * period):
            block = got[at:min(n, at + 64 * period)]
            whole = len(block) // period * period
            assert (block[:whole].view(-1, period, got.shape[1]) == part).all(), at
            assert torch.equal(block[whole:], part[:len(block) - whole]), at
        assert (got[n] == 0xA5).all()


@pytest.mark.parametrize("n,c", [(2, 16416), (1, 24576), (193, 16416), (131, 24576)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_three_chunks_of_1024_threads(dqm, n, c, dtype):
    x, r = _stream_rows(n, c, dtype, c + n), 2 * _stream_rows(n, c, dtype, c + n + 1)
    codes, scales, h, y = _outputs(n, c, dtype)
    dqm.dq_rmsnorm8(x.to(DEV), None, 1e-6, codes, scales, residual=r.to(DEV), h=h, y=y)
    _compare(rows.rms_norm8(_f32(x), _f32(r), None, 1e-6, dtype), codes, scales, h, y, dtype)


@pytest.mark.parametrize("n,ci,co,rank", [(1, 640, 8200, 40), (1, 1792, 8193, 64), (2, 640, 8208, 33), (4, 640, 8201, 64), (3, 96, 9000, 50)])
@pytest.mark.parametrize("kind", ["bf16", "f32", "mx8"])
def test_direct_product_with_more_ranks_and_many_channels(dqm, n, ci, co, rank, kind):
    _say(f"rows {n} {ci}->{co} rank {rank} {kind}")
    w, rc, rs, l1, l2 = _weight(dqm, ci, co, rank, n + ci + co)
    args, x64 = _x(n, ci, kind, n)
    for ytype in ("f32", "bf16"):
        y = torch.full((n + 1, co), float("nan"), dtype=TYPES[ytype], device=DEV)
        _call(dqm, w, args, dqm.dq_rows_create(w, n), y[:n])
        _check(y[:n], x64, rc, rs, l1, l2, 3 if kind == "f32" else 1, ytype)
        assert torch.isnan(y[n]).all()
