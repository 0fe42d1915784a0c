"""A device that is not there is refused the same way by every entry point that
takes one, before anything is read or written."""
import ctypes

import numpy as np
import pytest

from conftest import gpu_available

A16 = 1 << 20            # an address that is never followed


def _calls(lib, device):
    h = ctypes.c_void_p()
    out = ctypes.byref(h)
    w = np.zeros((32, 256), np.float32)
    perm, codes, scales = np.arange(256, dtype=np.int32), np.zeros((32, 128), np.uint8), np.zeros((32, 8), np.uint8)
    p = lambda a: ctypes.c_void_p(a.ctypes.data)
    yield "dq_prepare_weights", lib.dq_prepare_weights(p(w), 0, 256, 32, 0, 1, device, out)
    yield "dq_prepare_weights_lowrank", lib.dq_prepare_weights_lowrank(p(w), 0, 256, 32, 0, None, None, device, out)
    yield "dq_prepare_weights_w6", lib.dq_prepare_weights_w6(p(w), 0, 256, 32, 0, None, None, 2, device, out)
    yield "dq_orbit_prepare", lib.dq_orbit_prepare(p(w), 0, 256, 32, p(perm), 4, 4, device, out)
    yield "dq_import_weights", lib.dq_import_weights(p(codes), p(scales), 256, 32, 0, None, None, device, out)
    yield "dq_rmsnorm8", lib.dq_rmsnorm8(A16, 64, None, 0, 1, None, 0, 1e-6, 1, 64, 32, None, 0, 2 * A16, 3 * A16, None, 0, device, None)
    assert not h.value


def _refused(lib, device):
    for name, status in _calls(lib, device):
        said = lib.dq_last_error().decode()
        yield name, status, said


@pytest.mark.skipif(gpu_available(), reason="checks a machine without a GPU")
def test_no_device_at_all(lib):
    got = list(_refused(lib, 0))
    assert len(got) == 6 and all(status == 5 and "no HIP device" in said for _, status, said in got), got


@pytest.mark.gpu
@pytest.mark.parametrize("device", [-1, 63, 64, 1 << 30])
def test_index_out_of_range(lib, device):
    got = list(_refused(lib, device))
    assert len(got) == 6 and all(status == 1 and "device index out of range" in said for _, status, said in got), got
