"""The ends of the stated range of few-row products: MX-FP8 values are exact
below 2^128 and infinite from there (their few significant bits leave nothing
between 1.875 2^127 and 2^128), fp32 rows are exact up to the largest, and so are
weights; a coded weight of 2^128 or more is refused.  One channel of a row and
of an output's weights is not zero, so each output is one product and has no
rounding."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import mx
from parity_util import DEV

CI, CO = 160, 70
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


@pytest.fixture(scope="module")
def dqm(lib):
    from w4a4_quantized_linear_cube_amd import dq
    return dq


def _weights(dqm, at, codes, scale):
    """Channel `at` of output j holds code codes[j]; every other weight is zero."""
    rc = np.zeros((CO, CI // 2), np.uint8)
    rc[:, at // 2] = codes << (4 * (at % 2))
    return dqm.dq_import_weights(rc, np.full((CO, CI // 32), scale, np.uint8), None, None)


def _ends(v):
    """Finite below 2^128, infinite with v's sign from there."""
    return np.where(np.abs(v) < 2.0 ** 128, v, np.copysign(np.inf, v))


@pytest.mark.parametrize("scale", [0, 252, 253, 254])
@pytest.mark.parametrize("at", [0, 31, 95])
def test_weights_past_fp32_are_refused(lib, scale, at):
    """A weight of 2^128 or more has no value in bf16 or fp32: refused with its
    place; all below go on to the device (or to there being none)."""
    P = lambda a: ctypes.c_void_p(a.ctypes.data)
    h = ctypes.c_void_p()
    for code in range(16):
        codes, scales = np.full((3, 48), 0x33, np.uint8), np.full((3, 3), 127, np.uint8)
        codes[2, at // 32 * 16:at // 32 * 16 + 16] = 0
        codes[2, at // 2] = code << (4 * (at % 2))
        scales[2, at // 32] = scale
        status = lib.dq_import_weights(P(codes), P(scales), 96, 3, 0, None, None, 0, ctypes.byref(h))
        said = lib.dq_last_error().decode()
        if GRID[code & 7] * 2.0 ** (scale - 127) >= 2.0 ** 128:
            assert status == 1 and "2^128" in said and f"output 2, channel {at}" in said, (code, said)
        else:
            assert status in (0, 5), (code, said)
            lib.dq_weights_destroy(h)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 3, 16, 40])
@pytest.mark.parametrize("scale", [251, 252, 253, 254])
def test_largest_mx8_values(dqm, n, scale):
    one = np.full(CO, 2)                                       # E2M1 code of 1
    w = _weights(dqm, 37, one, 127)
    for first in range(0, 256, n):
        code = (np.arange(first, first + n) % 256).astype(np.uint8)
        codes = np.zeros((n, CI), np.uint8)
        codes[:, 37] = code
        y = torch.full((n, CO), 5.0, device=DEV)
        dqm.dq_linear_rows8(w, torch.from_numpy(codes).to(DEV), torch.full((n, CI // 32), scale, dtype=torch.uint8, device=DEV),
                            dqm.dq_rows_create(w, n), y)
        nan = (code & 0x7F) == 0x7F
        want = np.array([0.0 if k else float(mx.fp8_decode_magnitude(int(c & 0x7F))) * (-1.0) ** (c >> 7) for k, c in zip(nan, code)])
        want = _ends(want * 2.0 ** (scale - 127))
        got = y.double().cpu().numpy()
        assert np.isnan(got[nan]).all()
        assert np.array_equal(got[~nan], np.repeat(want[~nan, None], CO, axis=1)), (first, scale)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 3, 16, 40])
@pytest.mark.parametrize("scale", [252, 253, 254])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_largest_weights(dqm, n, scale, dtype):
    code = np.arange(CO) % 16
    code = np.where(GRID[code & 7] * 2.0 ** (scale - 127) < 2.0 ** 128, code, code & 8 | 3)
    w = _weights(dqm, 100, code, scale)
    x = np.zeros((n, CI), np.float32)
    x[:, 100] = 2.0 ** -(1.0 + np.arange(n) % 20)
    y = torch.empty(n, CO, device=DEV)
    dqm.dq_linear_rows(w, torch.from_numpy(x).to(torch.bfloat16 if dtype == "bf16" else torch.float32).to(DEV), dqm.dq_rows_create(w, n), y)
    want = GRID[code & 7] * np.where(code & 8, -1.0, 1.0) * 2.0 ** (scale - 127)
    assert np.array_equal(y.double().cpu().numpy(), x[:, 100:101] * want)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 3, 16, 40])
def test_largest_fp32_rows(dqm, n):
    w = _weights(dqm, 3, np.where(np.arange(CO) % 2, 2, 10), 127)          # +1 and -1
    big = np.float32([np.finfo(np.float32).max, -np.finfo(np.float32).max, 2.0 ** 127, np.nextafter(np.float32(2.0 ** 127), np.float32(0))])
    x = np.zeros((n, CI), np.float32)
    x[:, 3] = big[np.arange(n) % 4]
    y = torch.empty(n, CO, device=DEV)
    dqm.dq_linear_rows(w, torch.from_numpy(x).to(DEV), dqm.dq_rows_create(w, n), y)
    assert np.array_equal(y.cpu().numpy(), x[:, 3:4] * np.where(np.arange(CO) % 2, 1, -1).astype(np.float32))
