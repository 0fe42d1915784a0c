"""Helpers of the tests of heads: random caches, batches and rows."""
import numpy as np
import torch

from oracle import heads

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def stream_rows(n, c, dtype, seed, spread=0.7):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, c, generator=g) * torch.exp(spread * torch.randn(c, generator=g))
    x[:, torch.randint(0, c, (max(1, c // 256),), generator=g)] *= 20.0
    return x.to(TYPES[dtype])


def f32(t):
    return t.detach().float().cpu().numpy()


def bits(t):
    t = t.detach().cpu()
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).numpy()


def same_bits(got, want32, dtype):
    """A tensor against fp32 values rounded once to its type; NaN equals NaN."""
    want = torch.from_numpy(np.ascontiguousarray(want32)).to(TYPES[dtype])
    got = got.detach().cpu()
    nan = torch.isnan(want)
    assert torch.equal(nan, torch.isnan(got)), "NaN in other places"
    a, b = bits(torch.where(nan, 0, got)), bits(torch.where(nan, 0, want))
    assert np.array_equal(a, b), f"{(a != b).sum()} of {a.size} values differ"


class Batch:
    """A ragged batch and its pages, on the host and on a GPU: rows[b] rows of a sequence of length[b] tokens."""

    def __init__(self, rows, length, page_tokens, device, seed=0, spare=2, tail=0):
        self.first = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        self.length = np.asarray(length, np.int32)
        self.n = int(self.first[-1]) + tail
        need = [-(-int(l) // page_tokens) for l in length]
        self.count = max(1, sum(need) + spare)
        order = np.random.default_rng(seed).permutation(self.count)
        # (what lies behind a sequence's last page is never looked at: it names no page)
        self.pages = np.full((len(rows), max(1, max(need))), 2 ** 30, np.int32)
        for b, k in enumerate(need):
            self.pages[b, :k], order = order[:k], order[k:]
        self.P, self.device = page_tokens, device

    def seqs(self, dq):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(self.device)
        return dq.Seqs(t(self.first), t(self.length), t(self.pages))


def host_cache(batch, kv_heads, dim, nbits, seed, dtype=np.float32):
    """Random codes: (k_codes, k_scales, v_codes, v_scales) as numpy arrays."""
    g = np.random.default_rng(seed)
    out = []
    size = np.exp(0.5 * g.standard_normal(dim))
    for key in (True, False):
        v = g.standard_normal((batch.count, kv_heads, batch.P, dim))
        v = v * size if key else v + 0.5 * size
        out += heads.encode(v.astype(np.float32), nbits)
    return out


def device_cache(dq, arrays, device):
    t = [torch.from_numpy(np.ascontiguousarray(a)).to(device) for a in arrays]
    return dq.KV(*t)


def attend_all(q, batch, cache, nbits, kv_heads, dim, dtype, block=1, window=0, prefix=None, cap=0.0, scale=None):
    """(y, bound) fp64 [n][heads * dim] of all rows by the definition; q: tensor
    [n][heads * dim].  The bound:
      scores     D + 8 fp32 additions and roundings of terms of size scale sum |q| |k|,
                 4 roundings of a number of the score's size (the base-2 factor, the
                 maximum's subtraction) and 2^-21 of the exponential; with a cap 4
                 roundings of its size: e, a weight's relative error, twice (its sum's too)
      bf16       each weight rounded (2^-8), in the sum as in the product: off by
                 2^-8 sum w |v - y| <= 2^-7 sum w |v|; then y (2^-8)
      fp32       a weight's second part rounded: 2^-16, and y 2^-24
      sums       one fp32 rounding for each of L tokens, and 16 of joining
    """
    q64 = q.detach().double().cpu().numpy()
    n, c = q64.shape
    G = c // (kv_heads * dim)
    scale = dim ** -0.5 if scale is None else scale
    kd, vd = heads.decode(*cache[:2], nbits), heads.decode(*cache[2:], nbits)
    y, bound = np.zeros((n, c)), np.zeros((n, c))
    for b in range(len(batch.length)):
        L = int(batch.length[b])
        pg = np.array([heads.page_of(batch.pages, batch.count, batch.P, b, t) for t in range(L)], np.int64)
        have = pg >= 0
        place = np.arange(L) % batch.P
        for i in range(batch.first[b], min(batch.first[b + 1], n)):
            t = L - int(batch.first[b + 1]) + i
            on = heads.visible(t, L, block, window, 0 if prefix is None else int(prefix[b])) & have
            for h in range(kv_heads):
                s = slice(h * G * dim, (h + 1) * G * dim)
                out, size, qk, top = heads.attend(q64[i, s].reshape(G, dim), kd[pg, h, place], vd[pg, h, place], on, scale, cap)
                e = (dim + 8) * 2.0 ** -24 * qk + 6 * 2.0 ** -24 * top + 2.0 ** -21 + 4 * 2.0 ** -24 * cap
                e = 2 * e + (L + 16) * 2.0 ** -24
                e = (e + 2.0 ** -7) * size + 2.0 ** -8 * np.abs(out) if dtype == "bf16" else (e + 2.0 ** -16) * size + 2.0 ** -24 * np.abs(out)
                y[i, s], bound[i, s] = out.reshape(-1), e.reshape(-1)
    return y, bound


def near(got, want, bound):
    """A tensor within `bound` of fp64 values, NaN where they are."""
    got = got.detach().double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)), "NaN in other places"
    with np.errstate(invalid="ignore"):
        over = np.abs(got - want) - bound
    worst = np.nanmax(over) if over.size else -1.0
    assert worst <= 1e-37, f"{worst} over the bound, {np.nansum(over > 0)} of {over.size} values"
