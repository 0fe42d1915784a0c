"""dq_attn_rows where workgroups share the sequences' tokens: batches of up to 64
sequences and more, unequal lengths, several short tiles to a workgroup, parts
that see nothing, and the page tables and masks that move the shares' borders."""
import numpy as np
import pytest
import torch

from heads_util import Batch, TYPES, attend_all, device_cache, host_cache, near
from parity_util import DEV, _say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dqm(lib):
    from w4a4_quantized_linear_cube_amd import dq
    return dq


def _check(dqm, batch, kv_heads, group, dim, dtype, nbits=8, seed=1, prefix=None, **how):
    cache = host_cache(batch, kv_heads, dim, nbits, seed)
    kv, seqs = device_cache(dqm, cache, DEV), batch.seqs(dqm)
    q = (1.5 * torch.randn(batch.n, kv_heads * group * dim, generator=torch.Generator().manual_seed(seed + 1))).to(TYPES[dtype])
    y = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    pre = None if prefix is None else torch.from_numpy(np.asarray(prefix, np.int32)).to(DEV)
    dqm.dq_attn_rows(kv, seqs, q.to(DEV), dqm.dq_attn_create(0), y, prefix=pre, **how)
    want, bound = attend_all(q, batch, cache, nbits, kv_heads, dim, dtype, prefix=prefix, **how)
    rows = int(batch.first[-1])
    near(y[:rows], want[:rows], bound[:rows])
    assert (y[rows:] == 7).all()


# 64 sequences are one launch, 65 two, 130 three; few and many heads (whole tiles from 12 workgroups a head on)
@pytest.mark.parametrize("n", [2, 63, 64, 65, 130])
@pytest.mark.parametrize("kv_heads,group", [(1, 1), (2, 5), (16, 1)])
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("f32", 64)])
def test_many_sequences(dqm, n, kv_heads, group, dtype, dim):
    _say(f"shares {n} sequences, {kv_heads} x {group} x {dim} {dtype}")
    g = np.random.default_rng(n + kv_heads)
    length = g.integers(0, 90, n)
    length[n // 2] = 700
    rows = g.integers(0, 3, n)
    _check(dqm, Batch(rows.tolist(), length.tolist(), 16, DEV, seed=n, tail=1), kv_heads, group, dim, dtype, seed=n)


@pytest.mark.parametrize("rows", [1, 5, 20, 45])
def test_several_tiles_of_one_sequence(dqm, rows):
    """Up to 32 rows times heads to a tile, so that one sequence has many, each in parts."""
    _check(dqm, Batch([rows, 1], [900, 300], 32, DEV, seed=rows), 2, 7, 64, "bf16", seed=rows)
    _check(dqm, Batch([rows, 1], [900, 300], 32, DEV, seed=rows), 1, 3, 128, "f32", seed=rows)


@pytest.mark.parametrize("how", [dict(block=1, window=40, prefix=[70, 0, 33]), dict(block=16, window=64), dict(block=1, window=900),
                                 dict(block=1, prefix=[2000, 5, 0]), dict(block=0), dict(block=64, window=1, prefix=[1, 1, 1])], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masks_of_long_sequences(dqm, how, dtype):
    _check(dqm, Batch([40, 3, 1], [2000, 1100, 64], 64, DEV, seed=11), 1, 2, 64, dtype, seed=13, **how)


# parts of whole shares of the least size and of larger ones, and parts that cross from tile to tile (the more of them
# the more sequences, heads and tokens); 769 tokens are one block past what a workgroup takes without a join
@pytest.mark.parametrize("n,longest", [(1, 769), (5, 1100), (33, 800), (64, 1500), (64, 3000), (66, 900)])
@pytest.mark.parametrize("kv_heads,group,dim,dtype", [(1, 3, 128, "bf16"), (8, 2, 64, "bf16"), (8, 1, 64, "f32")])
def test_parts_of_tiles(dqm, n, longest, kv_heads, group, dim, dtype):
    _say(f"parts {n} sequences of up to {longest}, {kv_heads} x {group} x {dim} {dtype}")
    g = np.random.default_rng(n + longest)
    length = g.integers(longest // 4, longest + 1, n)
    length[0] = longest
    rows = g.integers(0, 2, n)
    rows[0] = 2
    _check(dqm, Batch(rows.tolist(), length.tolist(), 64, DEV, seed=n, tail=1), kv_heads, group, dim, dtype, seed=n)


def test_a_long_sequence_beside_short_ones(dqm):
    length = [5000] + [1] * 20 + [33] * 20
    _check(dqm, Batch([1] * 41, length, 64, DEV, seed=15), 1, 4, 64, "bf16", seed=17)


def test_nothing_cached(dqm):
    """Rows of empty sequences in a batch whose table is wide enough to be shared."""
    batch = Batch([2, 3, 0, 1], [0, 1, 0, 600], 16, DEV, seed=19)
    _check(dqm, batch, 2, 2, 64, "bf16", seed=21)
    batch = Batch([2, 3], [0, 0], 16, DEV, seed=23)
    batch.pages = np.zeros((2, 50), np.int32)
    _check(dqm, batch, 2, 2, 64, "f32", seed=25)


def test_the_workspace_keeps_nothing(dqm):
    """Calls of other shapes through one workspace leave nothing that a later one reads."""
    work = dqm.dq_attn_create(0)
    calls = []
    for i, (rows, length, heads, group, dim, dtype) in enumerate([([1] * 64, [50 * j + 1 for j in range(64)], 1, 2, 64, "bf16"),
                                                                  ([1], [3000], 2, 1, 128, "f32"), ([30], [400], 1, 2, 64, "bf16"),
                                                                  ([1, 1], [10, 2000], 4, 4, 64, "f32")]):
        batch = Batch(rows, length, 32, DEV, seed=30 + i)
        kv, seqs = device_cache(dqm, host_cache(batch, heads, dim, 8, 40 + i), DEV), batch.seqs(dqm)
        q = torch.randn(batch.n, heads * group * dim, generator=torch.Generator().manual_seed(50 + i)).to(TYPES[dtype]).to(DEV)
        alone = torch.empty_like(q)
        dqm.dq_attn_rows(kv, seqs, q, dqm.dq_attn_create(0), alone)
        calls.append((kv, seqs, q, alone))
    for _ in range(3):
        for kv, seqs, q, alone in calls:
            y = torch.empty_like(q)
            dqm.dq_attn_rows(kv, seqs, q, work, y)
            assert torch.equal(y, alone)


def test_two_workspaces_on_two_streams(dqm):
    batch = Batch([1, 1], [3000, 2000], 64, DEV, seed=61)
    kv, seqs = device_cache(dqm, host_cache(batch, 2, 64, 8, 63), DEV), batch.seqs(dqm)
    q = [torch.randn(2, 256, generator=torch.Generator().manual_seed(65 + i)).bfloat16().to(DEV) for i in range(2)]
    want = [torch.empty_like(x) for x in q]
    works = [dqm.dq_attn_create(0) for _ in range(2)]
    for i in range(2):
        dqm.dq_attn_rows(kv, seqs, q[i], works[i], want[i])
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [torch.zeros_like(x) for x in q]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            dqm.dq_attn_rows(kv, seqs, q[i], works[i], got[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_replays_while_lengths_grow(dqm):
    """Captured once, replayed as the lengths change, so that the shares' borders move; eager calls of the same between."""
    batch = Batch([1, 2, 1], [2500, 90, 700], 64, DEV, seed=71)
    kv, seqs = device_cache(dqm, host_cache(batch, 1, 128, 4, 73), DEV), batch.seqs(dqm)
    q = torch.randn(4, 640, generator=torch.Generator().manual_seed(75)).bfloat16().to(DEV)
    work, y, z = dqm.dq_attn_create(0), torch.zeros_like(q), torch.zeros_like(q)
    dqm.dq_attn_rows(kv, seqs, q, work, y)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        dqm.dq_attn_rows(kv, seqs, q, work, y)
    for step in (0, -3, -700, -30):
        seqs.tensors[1].add_(step).clamp_(min=0)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        dqm.dq_attn_rows(kv, seqs, q, work, z)
        assert torch.equal(y, z)
