"""dq_attn_rows where the sums of a sequence's tokens meet from several workgroups:
page tables of more than 768 tokens, whatever the lengths.  Equal scores over
values that mark blocks and tokens, whose sums and quotients are exact, so that
no token is left out or counted twice; and the masks, pages, extreme scores, caps
and NaN of shorter tables once more, against the definition."""
import numpy as np
import pytest
import torch

from heads_util import Batch, TYPES, attend_all, device_cache, host_cache, near
from oracle import heads
from parity_util import DEV, _say

WIDE = 1024                                          # tokens that a table has room for, at least


@pytest.fixture(scope="module")
def dqm(lib):
    from w4a4_quantized_linear_cube_amd import dq
    return dq


def _widen(batch, tokens=WIDE):
    """The batch with a page table for `tokens` tokens of each sequence; places past a sequence's own name no page."""
    more = -(-tokens // batch.P) - batch.pages.shape[1]
    if more > 0:
        batch.pages = np.ascontiguousarray(np.pad(batch.pages, ((0, 0), (0, more)), constant_values=2 ** 30))
    return batch


def _attend(dqm, batch, cache, q, prefix=None, work=None, **how):
    kv, seqs = device_cache(dqm, cache, DEV), batch.seqs(dqm)
    y = torch.full(q.shape, 7.0, dtype=q.dtype, device=DEV)
    pre = None if prefix is None else torch.from_numpy(np.asarray(prefix, np.int32)).to(DEV)
    dqm.dq_attn_rows(kv, seqs, q.to(DEV), work or dqm.dq_attn_create(0), y, prefix=pre, **how)
    return y


# ---------------------------------------------------------------------- marks ----
def _marks(L, dim):
    """[L][dim] of 0 and 1: channel c of the first half marks every (dim / 2)-th block of 32 tokens, of the second every (dim / 2)-th token."""
    t, c, half = np.arange(L)[:, None], np.arange(dim)[None], dim // 2
    return np.where(c < half, t // 32 % half == c, t % half == c - half)


def _shares(seen, dim):
    """fp32 [dim]: of the tokens `seen` [L] the share that each channel marks; zero of none."""
    n = np.float32(seen.sum())
    return (_marks(len(seen), dim) & seen[:, None]).sum(0).astype(np.float32) / n if n else np.zeros(dim, np.float32)


def _marked_cache(batch, kv_heads, dim, nbits):
    """Keys of zero, and in every page that holds tokens their marks (a code of 1.0), rolled by one channel for each head."""
    v = np.zeros((batch.count, kv_heads, batch.P, dim), np.uint8)
    for b, L in enumerate(batch.length):
        m = _marks(int(L), dim).astype(np.uint8) * (0x38 if nbits == 8 else 2)
        for i in range(min(-(-int(L) // batch.P), batch.pages.shape[1])):
            part = m[i * batch.P:(i + 1) * batch.P]
            if 0 <= batch.pages[b, i] < batch.count:
                for h in range(kv_heads):
                    v[batch.pages[b, i], h, :len(part)] = np.roll(part, h, axis=1)
    v = v if nbits == 8 else v[..., 0::2] | v[..., 1::2] << 4
    scales = np.full((*v.shape[:3], dim // 32), 127, np.uint8)
    return [np.zeros_like(v), scales, v, scales.copy()]


def _check_marks(dqm, batch, kv_heads, group, dim, dtype, nbits, prefix=None, **how):
    cache = _marked_cache(batch, kv_heads, dim, nbits)
    q = torch.randn(batch.n, kv_heads * group * dim, generator=torch.Generator().manual_seed(1)).to(TYPES[dtype])
    got = _attend(dqm, batch, cache, q, prefix, **how)
    want = np.full((batch.n, kv_heads, group, dim), 7.0, np.float32)
    for b, L in enumerate(batch.length.tolist()):
        have = np.array([heads.page_of(batch.pages, batch.count, batch.P, b, t) >= 0 for t in range(L)], bool)
        for i in range(batch.first[b], batch.first[b + 1]):
            on = heads.visible(L - int(batch.first[b + 1]) + i, L, how.get("block", 1), how.get("window", 0), 0 if prefix is None else prefix[b])
            share = _shares(on & have, dim)
            for h in range(kv_heads):
                want[i, h] = np.roll(share, h)
    want = torch.from_numpy(want.reshape(batch.n, -1)).to(TYPES[dtype]).to(DEV)
    assert torch.equal(got, want), f"{(got != want).sum().item()} of {got.numel()} values differ"


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("L", [1000, 20001])
def test_a_block_left_out_or_counted_twice_shows(dim, L):
    """On the CPU: every such mistake of one block of 32 tokens changes an fp32 answer, and of a whole one a bf16 answer.  (A
    channel marks at most 20 blocks at these lengths, so one of them is a twentieth of its share and more than the 2^-8 that
    bf16 rounds by; 20001's last block is a single token, 1 / 657 of its channels' shares, which only fp32 tells.)"""
    marks = _marks(L, dim)
    total = marks.sum(0)
    fp32 = lambda count, n: torch.from_numpy(count.astype(np.float32) / np.float32(n))
    good = fp32(total, L)
    assert np.array_equal(good.numpy(), _shares(np.ones(L, bool), dim))
    for i in range(0, L, 32):
        part = marks[i:i + 32].sum(0)
        n = min(32, L - i)
        for wrong in (fp32(total - part, L - n), fp32(total + part, L + n)):
            assert not torch.equal(wrong, good)
            assert n < 32 or not torch.equal(wrong.bfloat16(), good.bfloat16())


FORMS = [("bf16", 8, 128), ("bf16", 4, 128), ("f32", 8, 64), ("f32", 4, 128), ("bf16", 8, 64), ("bf16", 4, 64), ("f32", 8, 128), ("f32", 4, 64)]


# one sequence and few; 4 and more rows of 5 heads make blocks of 32 rows; a length just past a workgroup's, and long ones
@pytest.mark.gpu
@pytest.mark.parametrize("dtype,nbits,dim", FORMS)
@pytest.mark.parametrize("rows,length,page", [([1], [20001], 64), ([1, 2], [769, 9000], 32), ([8], [3000], 16), ([4, 0, 7], [2500, 0, 1100], 128),
                                              ([1], [257], 16), ([30], [5000], 256)])
def test_marks_of_long_sequences(dqm, dtype, nbits, dim, rows, length, page):
    _say(f"marks {rows} {length} page {page}, {dtype} {nbits} bits x {dim}")
    for kv_heads, group in ((1, 5), (2, 1), (5, 3)):
        _check_marks(dqm, _widen(Batch(rows, length, page, DEV, seed=3, tail=1)), kv_heads, group, dim, dtype, nbits)


# up to 64 sequences in one launch, more of them 64 at a time; with many heads the tiles fill the card by themselves
@pytest.mark.gpu
@pytest.mark.parametrize("dtype,nbits,dim", FORMS[:4])
@pytest.mark.parametrize("n,longest", [(9, 3000), (64, 1500), (65, 900), (130, 1200), (200, 800)])
@pytest.mark.parametrize("kv_heads", [1, 8])
def test_marks_of_ragged_batches(dqm, dtype, nbits, dim, n, longest, kv_heads):
    _say(f"marks of {n} sequences of up to {longest}, {kv_heads} heads, {dtype} {nbits} bits x {dim}")
    g = np.random.default_rng(n + longest + kv_heads)
    length = g.integers(0, longest + 1, n)
    length[n // 2] = longest
    rows = g.integers(0, 3, n)
    _check_marks(dqm, _widen(Batch(rows.tolist(), length.tolist(), 64, DEV, seed=n)), kv_heads, 2, dim, dtype, nbits)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,nbits,dim", FORMS[:4])
def test_marks_of_one_long_sequence_in_a_full_card(dqm, dtype, nbits, dim):
    """Tiles that fill the card are not shared: the long one is one workgroup's."""
    batch = _widen(Batch([1] * 100, [7000] + [40 + i for i in range(99)], 64, DEV, seed=5))
    _check_marks(dqm, batch, 8, 1, dim, dtype, nbits)
    batch = _widen(Batch([1] * 20, [40 + i for i in range(19)] + [7000], 64, DEV, seed=7))
    _check_marks(dqm, batch, 40, 1, dim, dtype, nbits)


MASKS = [dict(block=0), dict(block=1, window=700), dict(block=1, window=33, prefix=[500, 0, 70]), dict(block=64, window=640, prefix=[1, 1500, 32]),
         dict(block=500), dict(block=1, window=1, prefix=[1999, 0, 31])]


@pytest.mark.gpu
@pytest.mark.parametrize("how", MASKS, ids=str)
@pytest.mark.parametrize("dtype,nbits,dim", FORMS[:4])
def test_marks_under_masks(dqm, how, dtype, nbits, dim):
    _check_marks(dqm, _widen(Batch([40, 3, 1], [2000, 1500, 64], 64, DEV, seed=11)), 2, 2, dim, dtype, nbits, **how)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,nbits,dim", FORMS[:4])
def test_marks_around_bad_pages(dqm, dtype, nbits, dim):
    batch = _widen(Batch([2, 1, 3], [3000, 900, 1000], 16, DEV, seed=13))
    batch.pages[0, 5:40], batch.pages[0, 100], batch.pages[1, :] = -5, batch.count, 2 ** 30
    batch.pages[2, 0], batch.pages[2, 62] = -1, -2 ** 31
    _check_marks(dqm, batch, 2, 3, dim, dtype, nbits)
    batch.pages = np.ascontiguousarray(batch.pages[:, :80])          # tokens past the table
    _check_marks(dqm, batch, 2, 3, dim, dtype, nbits, block=0)


@pytest.mark.gpu
def test_marks_while_other_work_goes_through_the_workspace(dqm):
    """A call between that is shared as well, of other heads, rows and lengths."""
    work = dqm.dq_attn_create(0)
    batch, other = _widen(Batch([1, 2], [9001, 4000], 64, DEV, seed=15)), _widen(Batch([1] * 40, [2000 - 20 * i for i in range(40)], 16, DEV, seed=17))
    for _ in range(3):
        _check_marks(dqm, batch, 2, 3, 128, "bf16", 4, work=work)
        _check_marks(dqm, other, 1, 2, 64, "f32", 8, work=work)


# ----------------------------------------------------- against the definition ----
def _check(dqm, batch, nbits, kv_heads, group, dim, dtype, seed, cache=None, q=None, prefix=None, **how):
    cache = cache or host_cache(batch, kv_heads, dim, nbits, seed)
    q = (1.5 * torch.randn(batch.n, kv_heads * group * dim, generator=torch.Generator().manual_seed(seed + 1))).to(TYPES[dtype]) if q is None else q
    y = _attend(dqm, batch, cache, q, prefix, **how)
    want, bound = attend_all(q, batch, cache, nbits, kv_heads, dim, dtype, prefix=prefix, **how)
    rows = int(batch.first[-1])
    near(y[:rows], want[:rows], bound[:rows])
    assert (y[rows:] == 7).all()
    return y


@pytest.mark.gpu
@pytest.mark.parametrize("how", [dict(cap=2.0), dict(block=0, cap=30.0, scale=1.0), dict(window=500, prefix=[90, 0, 33], cap=5.0), dict(block=7, scale=0.3)], ids=str)
@pytest.mark.parametrize("dtype,nbits,dim", FORMS[:4])
def test_caps_and_masks(dqm, how, dtype, nbits, dim):
    _check(dqm, _widen(Batch([9, 1, 40], [1500, 800, 333], 16, DEV, seed=19, tail=1)), nbits, 2, 2, dim, dtype, 21, **how)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [63, 130])
@pytest.mark.parametrize("dtype,nbits,dim", [("bf16", 4, 128), ("f32", 8, 64)])
def test_short_sequences_in_a_wide_table(dqm, n, dtype, nbits, dim):
    g = np.random.default_rng(n)
    length, rows = g.integers(0, 90, n), g.integers(0, 3, n)
    length[n // 2] = 900
    _check(dqm, _widen(Batch(rows.tolist(), length.tolist(), 16, DEV, seed=n, tail=1)), nbits, 2, 2, dim, dtype, n, cap=4.0 if n == 63 else 0.0)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_cached(dqm, dtype):
    _check(dqm, _widen(Batch([2, 3, 0, 1], [0, 1, 0, 600], 16, DEV, seed=23)), 8, 2, 2, 64, dtype, 25)
    _check(dqm, _widen(Batch([2, 3], [0, 0], 16, DEV, seed=27)), 8, 2, 2, 64, dtype, 29)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("slope", [0.0, 0.25, -0.25, 8.0, -8.0])
def test_maxima_far_apart(dqm, dtype, slope):
    """Scores that rise or fall from part to part, some parts' worth being nothing."""
    P, dim, L = 32, 64, 1500
    batch = Batch([3], [L], P, DEV, seed=31)
    k = np.zeros((batch.count, 1, P, dim), np.float32)
    for t in range(L):
        k[batch.pages[0, t // P], 0, t % P, 0] = slope * t
    v = np.random.default_rng(33).standard_normal(k.shape).astype(np.float32)
    q = torch.zeros(3, dim)
    q[:, 0] = torch.tensor([8.0, -8.0, 0.0])
    _check(dqm, batch, 8, 1, 1, dim, dtype, 35, cache=[*heads.encode(k, 8), *heads.encode(v, 8)], q=q.to(TYPES[dtype]))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_masked_and_seen(dqm, dtype):
    """NaN behind the last token, in free pages and in one seen token of one part: its own channel, or with a key's every one, of the rows that see it."""
    P, kv_heads, dim = 16, 2, 64
    batch = _widen(Batch([6, 3], [1005, 700], P, DEV, seed=37))
    cache = host_cache(batch, kv_heads, dim, 8, 39)
    clean = _check(dqm, batch, 8, kv_heads, 2, dim, dtype, 41, cache=cache)
    used = np.zeros((batch.count, P), bool)
    for b in range(2):
        for t in range(batch.length[b]):
            used[batch.pages[b, t // P], t % P] = True
    for page, place in zip(*np.nonzero(~used)):
        for a, bad in zip(cache, (0x7F, 255, 0xFF, 255)):
            a[page, :, place] = bad
    assert torch.equal(_check(dqm, batch, 8, kv_heads, 2, dim, dtype, 41, cache=cache), clean)
    for t, first in ((1003, 4), (300, 0)):
        page, place = batch.pages[0, t // P], t % P
        for which, code, count in ((0, 0x7F, 2 * dim), (2, 0xFF, 2)):
            again = [a.copy() for a in cache]
            again[which][page, 1, place, 5] = code
            y = _check(dqm, batch, 8, kv_heads, 2, dim, dtype, 41, cache=again)
            assert torch.isnan(y).sum() == (6 - first) * count and torch.isnan(y[first:6]).sum() == (6 - first) * count
