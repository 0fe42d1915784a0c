"""dq_attn_rows over values and keys that are infinite (scale codes of 247 and
more): every row that sees such a value answers with its infinity, wherever the
value lies in its tile and whatever its weight, and the other rows and channels
answer as if it were zero."""
import numpy as np
import pytest
import torch

from heads_util import Batch, TYPES, attend_all, device_cache, host_cache
from oracle import heads
from parity_util import DEV, _say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dqm(lib):
    from w4a4_quantized_linear_cube_amd import dq
    return dq


def _run(dqm, batch, cache, q, **how):
    kv, seqs = device_cache(dqm, cache, DEV), batch.seqs(dqm)
    y = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    dqm.dq_attn_rows(kv, seqs, q.to(DEV), dqm.dq_attn_create(0), y, **how)
    return y.double().cpu().numpy()


def _put(batch, cache, nbits, b, t, head, channel, sign):
    """Makes channel `channel` of the value of token t infinite, the rest of its group of 32 zero."""
    page, place = batch.pages[b, t // batch.P], t % batch.P
    group = channel // 32
    codes = cache[2][page, head, place].view()
    codes[group * 32 * nbits // 8:(group + 1) * 32 * nbits // 8] = 0
    if nbits == 8:
        codes[channel] = 0x7E | (0x80 if sign < 0 else 0)
    else:
        codes[channel // 2] |= (0x7 | (0x8 if sign < 0 else 0)) << (4 * (channel % 2))
    cache[3][page, head, place, group] = 254


def _check(dqm, batch, nbits, kv_heads, group, dim, dtype, put, seed, q=None, cache=None, **how):
    cache = cache or host_cache(batch, kv_heads, dim, nbits, seed)
    q = (1.5 * torch.randn(batch.n, kv_heads * group * dim, generator=torch.Generator().manual_seed(seed + 1))).to(TYPES[dtype]) if q is None else q
    zeros = [a.copy() for a in cache]                        # (the same, and the infinite values zero)
    extra = np.zeros((batch.n, kv_heads * group, dim, 2), bool)
    for b, t, head, channel, sign in put:
        _put(batch, cache, nbits, b, t, head, channel, sign)
        _put(batch, zeros, nbits, b, t, head, channel, sign)
        page, place = batch.pages[b, t // batch.P], t % batch.P
        zeros[2][page, head, place, channel // 32 * 32 * nbits // 8:(channel // 32 + 1) * 32 * nbits // 8] = 0
        L = int(batch.length[b])
        for i in range(batch.first[b], batch.first[b + 1]):
            on = heads.visible(L - int(batch.first[b + 1]) + i, L, how.get("block", 1), how.get("window", 0), 0)
            if on[t]:
                extra[i, head * group:(head + 1) * group, channel, int(sign < 0)] = True
    extra = extra.reshape(batch.n, -1, 2)
    y = _run(dqm, batch, cache, q, **how)
    want, bound = attend_all(q, batch, zeros, nbits, kv_heads, dim, dtype, **how)
    up, down = extra[..., 0], extra[..., 1]
    assert up.any() and (~up).any()
    assert (y[up & ~down] == np.inf).all() and (y[down & ~up] == -np.inf).all() and np.isnan(y[up & down]).all()
    rest = ~up & ~down
    assert (np.abs(y - want) <= bound)[rest].all()


# in blocks that every row sees and that few do, in the first and the last token, both signs in one channel and in two
PUT = [(0, 3, 0, 5, 1), (0, 40, 0, 5, -1), (0, 70, 1, 37, -1), (0, 199, 1, 63, 1), (0, 195, 0, 40, 1), (1, 0, 0, 0, -1), (1, 30, 1, 33, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nbits", [8, 4])
@pytest.mark.parametrize("rows,group,dim", [(7, 1, 64), (7, 2, 128), (20, 3, 64), (20, 2, 128)])
def test_infinite_values(dqm, dtype, nbits, rows, group, dim):
    _say(f"infinite {rows} x {group} x {dim} {dtype} {nbits} bits")
    batch = Batch([rows, 3], [200, 31], 16, DEV, seed=3)
    for how in (dict(), dict(block=0), dict(block=8, window=64)):
        _check(dqm, batch, nbits, 2, group, dim, dtype, PUT, 5, **how)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_a_cache_that_is_split(dqm, dtype):
    """Among several workgroups' tokens, joined by the second launch."""
    batch = Batch([2, 1], [4000, 1500], 64, DEV, seed=7)
    _check(dqm, batch, 8, 1, 3, 64, dtype, [(0, 5, 0, 9, 1), (0, 2222, 0, 40, -1), (0, 3999, 0, 50, 1), (1, 700, 0, 3, 1), (1, 900, 0, 3, -1)], 9)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("slope", [0.25, -0.25])
@pytest.mark.parametrize("L", [500, 3000])
def test_whatever_their_weight(dqm, dtype, slope, L):
    """Scores that rise or fall along the cache, so that most weights, and what a wave's and a workgroup's sums are worth, are 0 in fp32."""
    P, dim = 32, 64
    batch = Batch([2], [L], P, DEV, seed=11)
    k = np.zeros((batch.count, 1, P, dim), np.float32)
    for t in range(L):
        k[batch.pages[0, t // P], 0, t % P, 0] = slope * t
    v = np.random.default_rng(13).standard_normal(k.shape).astype(np.float32)
    cache = [*heads.encode(k, 8), *heads.encode(v, 8)]
    q = torch.zeros(2, dim)
    q[:, 0] = 8.0
    _check(dqm, batch, 8, 1, 1, dim, dtype, [(0, 1, 0, 4, 1), (0, L // 2, 0, 20, -1), (0, L - 2, 0, 50, 1)], 15, q=q.to(TYPES[dtype]), cache=cache)
