"""Heads between their projection and attention: norm and rotation, a paged cache
of coded keys and values, and attention of query rows over it.

None of them is named by the pages; the codes are those of the quantizer of
关键设计 4 (readings R5-R7).  Readings taken:
  H1  the norm is F2's, over a head's channels or the whole row's;
  H2  a pair is rotated in fp32, product by product: a' = fl(fl(a c) - fl(b s)),
      b' = fl(fl(a s) + fl(b c)), c and s the fp32 roundings of cos and sin of
      the fp64 product of position and frequency;
  H3  what is not finite does not enter a group's scale; it takes the E4M3 NaN
      code, and where the elements are E2M1, which has none, the group takes
      the E8M0 NaN code;
  H4  a row that sees no token is zero.
Plain numpy; norms as in F2, attention in fp64, unrounded.
"""
from __future__ import annotations

import numpy as np

from . import mx, rows


def table(freq, positions: int) -> np.ndarray:
    """(cos, sin) [positions][pairs][2] in fp32."""
    angle = np.arange(positions, dtype=np.float64)[:, None] * np.asarray(freq, dtype=np.float64)
    return np.stack([np.cos(angle), np.sin(angle)], axis=-1).astype(np.float32)


def rotate(v32, tables, pos, interleaved: bool) -> np.ndarray:
    """v [N][H][D] by positions pos [N][axes] (H2); a position outside of its table is NaN."""
    v = np.array(v32, dtype=np.float32)
    cs = []
    for i, t in enumerate(tables):
        p = np.asarray(pos)[:, i]
        inside = (p >= 0) & (p < t.shape[0])
        cs.append(np.where(inside[:, None, None], t[np.where(inside, p, 0)], np.float32(np.nan)))
    cs = np.concatenate(cs, axis=1)[:, None]                       # [N][1][P][2]
    c, s = cs[..., 0], cs[..., 1]
    P = c.shape[-1]
    ia, ib = (np.arange(P) * 2, np.arange(P) * 2 + 1) if interleaved else (np.arange(P), np.arange(P) + P)
    a, b = v[..., ia], v[..., ib]
    with np.errstate(all="ignore"):
        v[..., ia], v[..., ib] = a * c - b * s, a * s + b * c
    assert v.dtype == np.float32
    return v


def norm_rope(x32, heads: int, norm=None, gain=None, eps: float = 1e-6, tables=None, pos=None, interleaved=True) -> np.ndarray:
    """fp32 [N][H][D] (H1, H2)."""
    x32 = np.asarray(x32, dtype=np.float32)
    n, c = x32.shape
    v = x32.reshape(n, heads, c // heads)
    with np.errstate(all="ignore"):
        if norm == "head":
            v = rows.rms_norm(v, None, gain, eps, "f32")[1]
        elif norm == "row":
            v = rows.rms_norm(x32, None, gain, eps, "f32")[1].reshape(v.shape)
    return v if tables is None else rotate(v, tables, pos, interleaved)


def encode(v32, bits: int):
    """Codes and scale codes of v [..., D] (H3): one E4M3 code per byte, or E2M1 packed two to a byte."""
    v = np.asarray(v32, dtype=np.float32)
    bad = ~np.isfinite(v)
    codes, scales = mx.mx_quantize(np.where(bad, np.float32(0), v), "fp8" if bits == 8 else "fp4")
    if bits == 8:
        return np.where(bad, codes | 0x7F, codes).astype(np.uint8), scales
    return mx.pack_fp4(codes), np.where(bad.reshape(scales.shape + (32,)).any(-1), 255, scales).astype(np.uint8)


def decode(codes, scales, bits: int) -> np.ndarray:
    """fp64 values [..., D]."""
    codes = np.asarray(codes, dtype=np.uint8)
    el = mx.unpack_fp4(codes) if bits == 4 else codes
    nan = ((el & 0x7F) == 0x7F) if bits == 8 else np.zeros(el.shape, bool)
    v = mx.mx_dequantize(np.where(nan, 0, el), scales, "fp8" if bits == 8 else "fp4")
    nan = nan | np.repeat(np.asarray(scales) == 255, 32, axis=-1)
    return np.where(nan, np.nan, v)


def places(first, length, n: int):
    """Sequence of each of n rows (-1: none) and its place there."""
    b, t = np.full(n, -1), np.zeros(n, np.int64)
    for i in range(len(length)):
        r = np.arange(max(first[i], 0), min(first[i + 1], n))
        b[r] = i
        t[r] = length[i] - first[i + 1] + r
    return b, t


def page_of(pages, count: int, page_tokens: int, b: int, t: int) -> int:
    """The page that holds token t of sequence b, -1 if none does."""
    i = t // page_tokens
    if t < 0 or i >= pages.shape[1]:
        return -1
    return int(pages[b, i]) if 0 <= pages[b, i] < count else -1


def visible(t: int, length: int, block: int, window: int, prefix: int) -> np.ndarray:
    """Which of a sequence's tokens the row at place t sees, by the definition."""
    tok = np.arange(length)
    if block == 0:
        return np.ones(length, bool)
    end = (t // block + 1) * block
    on = tok < end
    if window:
        on &= tok >= end - window
    return on | (tok < prefix)


def attend(q64, k64, v64, on, scale: float, cap: float = 0.0):
    """One row's heads: q [G][D] over k, v [L][D], `on` [L].  (y [G][D]; sum w |v|
    [G][D]; the largest scale sum |q| |k| and the largest |score| of each head
    [G][1], that error bounds go by.)"""
    G, D = q64.shape
    if not on.any():
        return np.zeros((G, D)), np.zeros((G, D)), np.zeros((G, 1)), np.zeros((G, 1))
    k64, v64 = k64[on], v64[on]
    with np.errstate(all="ignore"):
        s = scale * (q64 @ k64.T)
        if cap:
            s = cap * np.tanh(s / cap)
        w = np.exp(s - s.max(axis=-1, keepdims=True))
        w = w / w.sum(axis=-1, keepdims=True)
        size = scale * (np.abs(q64) @ np.abs(k64).T)
        return w @ v64, w @ np.abs(v64), size.max(axis=-1, keepdims=True), np.abs(s).max(axis=-1, keepdims=True)
