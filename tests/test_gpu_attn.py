"""dq_attn_rows on the GPU against its definition in 64 bits, within a derived bound."""
import numpy as np
import pytest
import torch

from heads_util import Batch, TYPES, attend_all, device_cache, host_cache, near, stream_rows
from parity_util import DEV, _say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dqm(lib):
    from w4a4_quantized_linear_cube_amd import dq
    return dq


def _q(n, c, dtype, seed):
    return (1.5 * torch.randn(n, c, generator=torch.Generator().manual_seed(seed))).to(TYPES[dtype])


def _run(dqm, batch, cache, q, work=None, **how):
    kv, seqs = device_cache(dqm, cache, DEV), batch.seqs(dqm)
    y = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    p = how.pop("prefix", None)
    how["prefix"] = None if p is None else torch.from_numpy(np.asarray(p, np.int32)).to(DEV)
    dqm.dq_attn_rows(kv, seqs, q.to(DEV), work or dqm.dq_attn_create(0), y, **how)
    torch.cuda.synchronize()
    return y


def _check(dqm, batch, nbits, kv_heads, group, dim, dtype, seed=1, **how):
    cache = host_cache(batch, kv_heads, dim, nbits, seed)
    q = _q(batch.n, kv_heads * group * dim, dtype, seed + 1)
    y = _run(dqm, batch, cache, q, **how)
    want, bound = attend_all(q, batch, cache, nbits, kv_heads, dim, dtype, **how)
    rows = int(batch.first[-1])
    near(y[:rows], want[:rows], bound[:rows])
    assert (y[rows:] == 7).all()


# one token, lengths around a block of 32 tokens and a round of four, ragged batches, no rows, more rows than tokens
BATCHES = [([1], [1], 16), ([1], [31], 16), ([1], [33], 32), ([1, 1], [128, 129], 64), ([1] * 5, [1, 500, 77, 16, 17], 16),
           ([3, 0, 9, 1], [3, 5, 200, 33], 16), ([6, 2], [4, 9], 32), ([17], [700], 256), ([2], [0], 16), ([1] * 70, [3 * i + 1 for i in range(70)], 16)]


@pytest.mark.parametrize("rows,length,page", BATCHES)
@pytest.mark.parametrize("kv_heads,group,dim", [(2, 1, 64), (1, 5, 128), (3, 16, 64), (2, 8, 128)])
@pytest.mark.parametrize("dtype,nbits", [("bf16", 8), ("f32", 4), ("bf16", 4), ("f32", 8)])
def test_causal(dqm, rows, length, page, kv_heads, group, dim, dtype, nbits):
    _say(f"attn {rows[:4]} {length[:4]} page {page}, {kv_heads} x {group} x {dim} {dtype} {nbits} bits")
    _check(dqm, Batch(rows, length, page, DEV, seed=3, tail=2), nbits, kv_heads, group, dim, dtype, seed=len(rows) + dim)


MASKS = [dict(block=0), dict(block=4), dict(block=1, window=1), dict(block=1, window=50), dict(block=7, window=20), dict(block=1000),
         dict(block=1, window=10, prefix=[5, 0, 300, -3]), dict(block=3, window=64, prefix=[100, 33, 1, 64]),
         dict(block=1, prefix=[150, 0, 64, 7]), dict(block=1, cap=2.0), dict(block=0, cap=30.0, scale=1.0), dict(block=2 ** 31 - 1, window=2 ** 31 - 1)]


@pytest.mark.parametrize("how", MASKS, ids=str)
@pytest.mark.parametrize("dtype,nbits,dim", [("bf16", 8, 128), ("f32", 8, 64), ("bf16", 4, 64)])
def test_masks(dqm, how, dtype, nbits, dim):
    _check(dqm, Batch([9, 1, 40, 5], [150, 40, 333, 64], 16, DEV, seed=5), nbits, 2, 2, dim, dtype, seed=7, **how)


@pytest.mark.parametrize("dtype,group", [("bf16", 4), ("f32", 4), ("bf16", 1)])
def test_a_long_cache_is_split(dqm, dtype, group):
    """Many workgroups to a head, joined in order; the same bits each time, also with other work in the workspace between."""
    batch = Batch([1, 2], [20001, 9000], 64, DEV, seed=9)
    cache, work = host_cache(batch, 2, 64, 8, 11), dqm.dq_attn_create(0)
    q = _q(batch.n, 2 * group * 64, dtype, 13)
    y = _run(dqm, batch, cache, q, work)
    want, bound = attend_all(q, batch, cache, 8, 2, 64, dtype)
    near(y, want, bound)
    other = Batch([1] * 9, [700] * 9, 16, DEV, seed=15)
    for _ in range(3):
        _run(dqm, other, host_cache(other, 1, 128, 4, 17), _q(9, 128, "bf16", 19), work)
        assert torch.equal(_run(dqm, batch, cache, q, work), y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,group", [(16, 1), (17, 1), (33, 1), (70, 1), (3, 11), (1, 40)])
def test_blocks_of_rows(dqm, dtype, rows, group):
    """Up to 16, 32 and 64 rows times heads at a time, and more."""
    _check(dqm, Batch([rows], [200], 32, DEV, seed=21), 8, 1, group, 64, dtype, seed=23)


def test_what_masked_places_hold_has_no_effect(dqm):
    """NaN codes and scales behind the last token, in pages of others, under the mask; a visible one reaches exactly the rows that see it."""
    P, kv_heads, dim = 16, 2, 64
    for dtype in ("bf16", "f32"):
        batch = Batch([6, 3], [45, 21], P, DEV, seed=25)
        cache = host_cache(batch, kv_heads, dim, 8, 27)
        q = _q(batch.n, kv_heads * 2 * dim, dtype, 29)
        clean = _run(dqm, batch, cache, q)
        used = np.zeros((batch.count, P), bool)
        for b in range(2):
            for t in range(batch.length[b]):
                used[batch.pages[b, t // P], t % P] = True
        for page, place in zip(*np.nonzero(~used)):
            for a, bad in zip(cache, (0x7F, 255, 0xFF, 255)):
                a[page, :, place] = bad
        assert torch.equal(_run(dqm, batch, cache, q), clean)
        # the token of the second last row of the first sequence: seen by that row and the last one
        page, place = batch.pages[0, 43 // P], 43 % P
        for which, code in ((0, 0x7F), (2, 0xFF)):
            again = [a.copy() for a in cache]
            again[which][page, 1, place, 5] = code
            y = _run(dqm, batch, again, q)
            want, bound = attend_all(q, batch, again, 8, kv_heads, dim, dtype)
            near(y, want, bound)
            assert torch.isnan(y[4:6]).any() and not torch.isnan(y[:4]).any() and not torch.isnan(y[6:]).any()
            if which == 2:                                       # (a value's NaN stays in its channel)
                assert torch.isnan(y[4:6]).sum() == 4


def test_bad_pages_are_not_seen(dqm):
    batch = Batch([2, 1, 3], [100, 40, 20], 16, DEV, seed=31)
    batch.pages[0, 2], batch.pages[0, 3], batch.pages[1, :] = -5, batch.count, 2 ** 30
    batch.pages[2, 0] = -1
    _check(dqm, batch, 8, 2, 3, 64, "bf16", seed=33)
    batch.pages = np.ascontiguousarray(batch.pages[:, :3])       # tokens past the table
    _check(dqm, batch, 8, 2, 3, 64, "f32", seed=35)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extreme_scores(dqm, dtype):
    """Scores far apart, equal, and falling along the cache, so that the maximum moves from one end to the other."""
    P, dim, L = 32, 64, 400
    batch = Batch([3], [L], P, DEV, seed=37)
    from oracle import heads
    for slope in (0.0, 0.5, -0.5, 20.0, -20.0):
        k = np.zeros((batch.count, 1, P, dim), np.float32)
        for t in range(L):
            k[batch.pages[0, t // P], 0, t % P, 0] = slope * t
        v = np.random.default_rng(39).standard_normal(k.shape).astype(np.float32)
        cache = [*heads.encode(k, 8), *heads.encode(v, 8)]
        q = torch.zeros(3, dim)
        q[:, 0] = torch.tensor([8.0, -8.0, 0.0])
        q = q.to(TYPES[dtype])
        y = _run(dqm, batch, cache, q)
        want, bound = attend_all(q, batch, cache, 8, 1, dim, dtype)
        near(y, want, bound)


def test_infinite_queries_stay_in_their_rows(dqm):
    batch = Batch([4], [50], 16, DEV, seed=41)
    cache = host_cache(batch, 1, 64, 8, 43)
    for dtype in ("bf16", "f32"):
        q = _q(4, 128, dtype, 45)
        clean = _run(dqm, batch, cache, q)
        q[1, 3], q[2, 100] = float("inf"), float("nan")
        y = _run(dqm, batch, cache, q)
        assert torch.isnan(y[1, :64]).all() and torch.isnan(y[2, 64:]).all()
        for r, c in ((0, slice(None)), (3, slice(None)), (1, slice(64, None)), (2, slice(0, 64))):
            assert torch.equal(y[r, c], clean[r, c])


def test_strided_rows_and_a_stream(dqm):
    batch = Batch([3, 2], [77, 300], 16, DEV, seed=47)
    cache = host_cache(batch, 2, 128, 8, 49)
    kv, seqs, work = device_cache(dqm, cache, DEV), batch.seqs(dqm), dqm.dq_attn_create(0)
    c = 2 * 3 * 128
    q = _q(5, c, "bf16", 51)
    wide, out = torch.zeros(5, c + 24, dtype=torch.bfloat16, device=DEV), torch.full((5, 2 * c), 3.0, dtype=torch.bfloat16, device=DEV)
    wide[:, 8:8 + c] = q.to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dqm.dq_attn_rows(kv, seqs, wide[:, 8:8 + c], work, out[:, c:], stream=s)
    s.synchronize()
    assert torch.equal(out[:, c:], _run(dqm, batch, cache, q)) and (out[:, :c] == 3).all()


def test_a_decoding_step(dqm):
    """As a program uses them: projections of a few rows, heads normed and rotated
    and their keys and values cached, attention, the output projection; captured
    and replayed while the sequences grow, against eager steps on a copy."""
    from oracle import heads
    B, kv_heads, group, dim, P, steps = 3, 2, 2, 64, 16, 5
    c, qc = kv_heads * dim, kv_heads * group * dim
    width = qc + 2 * c
    g = torch.Generator().manual_seed(53)
    ci = 256
    w1 = dqm.dq_prepare_weights_lowrank(torch.randn(width, ci, generator=g) / 16, None, None)
    w2 = dqm.dq_prepare_weights_lowrank(torch.randn(ci, qc, generator=g) / 16, None, None)
    r1, r2, work = dqm.dq_rows_create(w1, B), dqm.dq_rows_create(w2, B), dqm.dq_attn_create(0)
    rope = dqm.Rope([torch.from_numpy(heads.table(10000.0 ** (-np.arange(dim // 2) / (dim // 2)), 64)).to(DEV)], False)
    batch = Batch([1] * B, [40 + steps, 7 + steps, 16 + steps], P, DEV, seed=55)     # (pages for what the steps add)
    batch.length = batch.length - steps
    start = host_cache(batch, kv_heads, dim, 8, 57)
    gain = (1 + 0.1 * torch.randn(dim, generator=g)).to(DEV)

    def program():
        kv, seqs = device_cache(dqm, start, DEV), batch.seqs(dqm)
        x, stacked = torch.zeros(B, ci, dtype=torch.bfloat16, device=DEV), torch.zeros(B, width, device=DEV)
        q, att, y = (torch.zeros(B, m, dtype=torch.bfloat16, device=DEV) for m in (qc, qc, ci))

        def step():
            seqs.tensors[1].add_(1)
            dqm.dq_linear_rows(w1, x, r1, stacked)
            dqm.dq_kv_write(kv, seqs, stacked[:, qc:qc + c], stacked[:, qc + c:], q=stacked[:, :qc], y=q, norm="head", gain=gain,
                            gain_q=gain, rope=rope)
            dqm.dq_attn_rows(kv, seqs, q, work, att)
            dqm.dq_linear_rows(w2, att, r2, y)
        return kv, seqs, x, q, att, y, step

    eager, captured = program(), program()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        captured[-1]()
    for i in range(steps):
        x = stream_rows(B, ci, "bf16", 60 + i).to(DEV)
        for p in (eager, captured):
            p[2].copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        eager[-1]()
        for a, b in zip((*eager[0].tensors, *eager[3:6]), (*captured[0].tensors, *captured[3:6])):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        # the attention's rows by the definition, from the cache as it stands
        now = Batch([1] * B, eager[1].tensors[1].cpu().numpy(), P, DEV, seed=55)
        now.pages, now.count = batch.pages, batch.count
        want, bound = attend_all(eager[3], now, [t.cpu().numpy() for t in eager[0].tensors], 8, kv_heads, dim, "bf16")
        near(eager[4], want, bound)


def test_a_cache_past_32_bits(dqm):
    """Pages whose codes lie past 2^32 bytes."""
    P, kv_heads, dim, L = 4096, 8, 128, 100
    pages = 2 ** 32 // (P * kv_heads * dim) + 2
    small = Batch([1], [L], P, DEV, seed=63, spare=0)
    cache = host_cache(small, kv_heads, dim, 8, 65)
    q = _q(1, 2 * kv_heads * dim, "bf16", 67)
    y = _run(dqm, small, cache, q)
    big = []
    for a in cache:
        t = torch.zeros(pages, *a.shape[1:], dtype=torch.uint8, device=DEV)
        t[pages - 1] = torch.from_numpy(a[small.pages[0, 0]]).to(DEV)
        big.append(t)
    kv = dqm.KV(*big)
    small.pages = np.array([[pages - 1]], np.int32)
    out = torch.empty_like(y)
    dqm.dq_attn_rows(kv, small.seqs(dqm), q.to(DEV), dqm.dq_attn_create(0), out)
    assert torch.equal(out, y)
