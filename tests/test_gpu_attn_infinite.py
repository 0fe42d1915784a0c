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


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nbits", [8, 4])
@pytest.mark.parametrize("rows,dim", [(5, 64), (20, 128)])
@pytest.mark.parametrize("cap", [0.0, 2.0])
def test_infinite_keys(dqm, dtype, nbits, rows, dim, cap):
    """A key's infinite channel: a score of the sign of its product with the query's.  Of -infinity the token has no
    weight, of +infinity none but NaN is the answer; capped scores are the cap.  (The queries' bits past bf16's are of either sign.)"""
    _say(f"infinite keys {rows} x {dim} {dtype} {nbits} bits cap {cap}")
    batch = Batch([rows], [200], 16, DEV, seed=17)
    cache = host_cache(batch, 1, dim, nbits, 19)
    q = (1.5 * torch.randn(rows, 2 * dim, generator=torch.Generator().manual_seed(21))).to(TYPES[dtype])
    q[0] = q[0].bfloat16().to(q.dtype)
    for t, channel, sign in ((7, 3, 1), (100, 40, -1), (199 - rows // 2, 3, 1)):
        page, place, group = batch.pages[0, t // 16], t % 16, channel // 32
        codes = cache[0][page, 0, place]
        codes[group * 32 * nbits // 8:(group + 1) * 32 * nbits // 8] = 0
        if nbits == 8:
            codes[channel] = 0x7E | (0x80 if sign < 0 else 0)
        else:
            codes[channel // 2] |= (0x7 | (0x8 if sign < 0 else 0)) << (4 * (channel % 2))
        cache[1][page, 0, place, group] = 254
    y = _run(dqm, batch, cache, q, cap=cap)
    # the definition, with an infinite score in the place of its product
    k, v = heads.decode(*cache[:2], nbits), heads.decode(*cache[2:], nbits)
    at = np.arange(200)
    k, v = k[batch.pages[0, at // 16], 0, at % 16], v[batch.pages[0, at // 16], 0, at % 16]
    finite = np.where(np.abs(k) < 2.0 ** 120, k, 0.0)
    seen = set()
    for i in range(rows):
        on = np.arange(200) <= 200 - rows + i
        for h in range(2):
            x = q[i, h * dim:(h + 1) * dim].double().numpy()
            far = np.where(np.abs(k) < 2.0 ** 120, 0.0, np.copysign(np.inf, k * x)).sum(axis=1)   # (one in a key at most)
            s = finite @ x * dim ** -0.5 + far
            got = y[i, h * dim:(h + 1) * dim]
            if cap:
                s = cap * np.tanh(s / cap)
            w = np.where(on, np.exp(s - s[on].max()), 0.0) if not (s[on] == np.inf).any() else None
            seen.add(w is None)
            if w is None:
                assert np.isnan(got).all()
                continue
            w = w / w.sum()
            # the bound of attend_all's, of the keys' finite part
            size = w @ np.abs(v)
            qk = (np.abs(finite) @ np.abs(x) * dim ** -0.5)[on].max()
            e = 2 * ((dim + 8) * 2.0 ** -24 * qk + 6 * 2.0 ** -24 * min(qk, cap or qk) + 2.0 ** -21 + 4 * 2.0 ** -24 * cap) + 216 * 2.0 ** -24
            e = (e + 2.0 ** -16) * size + (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) * np.abs(w @ v)
            assert (np.abs(got - w @ v) <= e).all()
    assert seen == ({False} if cap else {False, True})
