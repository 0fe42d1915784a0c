"""dq_attn_rows: a weight keeps its bits where it meets its value, whatever the rows' type."""
import numpy as np
import pytest
import torch

from heads_util import TYPES
from parity_util import DEV, _say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dqm(lib):
    from w4a4_quantized_linear_cube_amd import dq
    return dq


# rows that share a key head: one block of 16, and blocks of 32
@pytest.mark.parametrize("rows", [9, 160])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nbits", [8, 4])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_values_of_opposite_sign(dqm, dtype, nbits, dim, rows):
    """Two tokens, of scores 0 and -x and values 1 and -1, so y = (1 - p) / (1 + p) with p = exp(-x) = O(1): for small x a
    weight's rounding is all that is left.  Row n has x_n = q_n (scale 1) in [2^-10, 2^-4], exact in every product.

    With u = 2^-24: the exponent's argument, rounded twice (its factor log2 e, and the product), is off by 2 u x log2 e;
    the exponential by one step of fp32, 2 u; the weight's parts leave 2^-16 (bf16: two) or u (fp32: three); the sums of
    weights and of weighted values, the second over parts, one rounding each of 2 at most and one for each part, 4 u
    (bf16) or 6 u; each of these moves y by half of itself or less, as the denominator is at least 1.9 and |v| 1:
    0.53 of their sum.  The division and the type's own rounding follow: u |y| and 2^-8 |y| (bf16) or u |y|."""
    _say(f"opposite values {rows} x {dim} {dtype} {nbits} bits")
    one = 0x38 if nbits == 8 else 0x02                           # 1.0
    codes = lambda: np.zeros((1, 1, 16, dim * nbits // 8), np.uint8)
    k, v, scales = codes(), codes(), np.full((1, 1, 16, dim // 32), 127, np.uint8)
    k[0, 0, 1, 0] = one | (0x80 if nbits == 8 else 0x08)         # channel 0: -1
    if nbits == 8:
        v[0, 0, 0], v[0, 0, 1] = one, one | 0x80
    else:
        v[0, 0, 0], v[0, 0, 1] = 0x22, 0xAA
    t = lambda a: torch.from_numpy(a).to(DEV)
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)
    kv = dqm.KV(t(k), t(scales), t(v), t(scales.copy()))
    x = torch.from_numpy(np.exp2(np.linspace(-10, -4, rows))).to(TYPES[dtype])
    q = torch.zeros(rows, dim, dtype=x.dtype)
    q[:, 0] = x
    y = torch.empty_like(q, device=DEV)
    dqm.dq_attn_rows(kv, dqm.Seqs(i32(0, rows), i32(2), i32(0)[None]), q.to(DEV), dqm.dq_attn_create(0), y, scale=1.0, block=0)
    x = x.double().numpy()[:, None]
    want = -np.expm1(-x) / (1 + np.exp(-x))
    u = 2.0 ** -24
    error = 0.53 * (2 * u * x * 1.4427 + 2 * u + (2.0 ** -16 + 4 * u if dtype == "bf16" else u + 6 * u))
    error = error + (u + (2.0 ** -8 if dtype == "bf16" else 0.0)) * want
    over = np.abs(y.double().cpu().numpy() - want) - error
    assert over.max() <= 0, f"{over.max()} over the bound, {(over > 0).sum()} of {over.size} values"
