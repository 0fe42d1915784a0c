"""A row's norm does not depend on the rows beside it: the order of its sum of
squares goes by the number of channels alone.

eps is put where f = fl32(1 / sqrt(mean + eps)) lies next to the border of two
fp32 values, so that one unit in the last place of the fp64 mean can move f and
every value of the row with it."""
import numpy as np
import pytest
import torch

from oracle import rows
from parity_util import DEV, _say

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def sum_of_squares(h):
    """In the stated order: 8 channels one by one, and such chunks pairwise by the bits of their place."""
    h = np.asarray(h, np.float64)
    chunks = np.zeros(4096)
    for j in range(8):                                        # (a square of 24 bits is exact: one rounding for each)
        chunks[:len(h) // 8] += h[j::8] ** 2
    while len(chunks) > 1:
        chunks = chunks[0::2] + chunks[1::2]
    return float(chunks[0])


def border_eps(s, c, count):
    """`count` consecutive values of eps around the one that puts the mean on a border of f."""
    mean = s / c
    f = np.float32(1.0 / np.sqrt(mean * 1.001))
    border = (float(f) + float(np.nextafter(f, np.float32(0)))) / 2
    eps = 1.0 / border / border - mean
    step = np.spacing(mean + eps)                             # (smaller ones do not reach the sum)
    return [eps + (k - count // 2) * step for k in range(count)]


def values(h, s, eps):
    f = np.float32(1.0 / np.sqrt(s / len(h) + eps))
    return np.asarray(h, np.float32) * f


# widths that few and many rows take by different numbers of threads, and some that they do not
@pytest.mark.parametrize("c", [96, 512, 544, 1024, 1536, 2048, 2080, 5120, 8192, 8224, 13824, 16384, 16416])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_alone_and_among_many(lib, c, dtype):
    from w4a4_quantized_linear_cube_amd import dq
    _say(f"norm of one row of {c} alone and among many, {dtype}")
    many = (3 << 20) // c + 3
    g = torch.Generator().manual_seed(c)
    moved = 0
    for trial in range(4):
        row = (torch.randn(c, generator=g) * torch.exp(3 * torch.randn(c, generator=g))).to(TYPES[dtype])
        h = row.float().numpy()
        s = sum_of_squares(h)
        one, all_ = row[None].to(DEV), row.repeat(many, 1).to(DEV)
        ys = [torch.empty_like(t) for t in (one, all_)]
        codes, scales = ([torch.empty(t.shape[0], k, dtype=torch.uint8, device=DEV) for t in (one, all_)] for k in (c, c // 32))
        seen = set()
        for eps in border_eps(s, c, 10):
            for x, y, cc, sc in zip((one, all_), ys, codes, scales):
                dq.dq_rmsnorm8(x, None, eps, cc, sc, y=y)
            want = values(h, s, eps)
            seen.add(want.tobytes())
            assert torch.equal(ys[1], ys[0].expand_as(ys[1])) and torch.equal(codes[1], codes[0].expand_as(codes[1])), (trial, eps)
            assert torch.equal(scales[1], scales[0].expand_as(scales[1])), (trial, eps)
            assert np.array_equal(ys[0][0].float().cpu().numpy(), rows.to_stream(want, dtype)), (trial, eps)
        moved += len(seen) > 1
    assert moved >= 3                                         # (the borders were met)
