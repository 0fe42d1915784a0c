"""Few-row operators: the residual RMS norm with MX-FP8 output, and products
of a few rows with a 4-bit weight.

Neither is named by the pages; both are built from the quantizer of 关键设计 4
(readings R5-R7) and its weight split W = L1 L2 + R.  Readings taken:
  F1  the norm is that of the residual stream as it is stored: h = x + r in
      fp32, rounded to the stream's type;
  F2  f = fl32(1 / sqrt(mean(h^2) + eps)) formed in fp64, then one fp32
      rounding for h f and one for its product with the gain;
  F3  the low-rank branch of a product is (x L1) L2 in the product's own
      precision: U is not rounded to bf16 as in R10.
Plain numpy; products in fp64, unrounded.
"""
from __future__ import annotations

import numpy as np

from . import mx


def to_stream(v32: np.ndarray, dtype: str) -> np.ndarray:
    """fp32 values rounded to the stream's type ("bf16" or "f32"), as fp32."""
    v32 = np.asarray(v32, dtype=np.float32)
    return v32 if dtype == "f32" else mx.bf16_bits_to_f64(mx.f32_to_bf16_bits(v32)).astype(np.float32)


def rms_norm(x32, r32, gain32, eps: float, dtype: str):
    """(h, v), both fp32 arrays: the stream after the addition (F1) and the normalized values (F2)."""
    x32 = np.asarray(x32, dtype=np.float32)
    h = x32 if r32 is None else to_stream(x32 + np.asarray(r32, dtype=np.float32), dtype)
    mean = (h.astype(np.float64) ** 2).sum(axis=-1, keepdims=True) / h.shape[-1]
    f = (1.0 / np.sqrt(mean + eps)).astype(np.float32)
    v = h * f
    if gain32 is not None:
        v = v * np.asarray(gain32, dtype=np.float32)
    assert v.dtype == np.float32
    return h, v


def rms_norm8(x32, r32, gain32, eps: float, dtype: str, group: int = 32) -> dict:
    h, v = rms_norm(x32, r32, gain32, eps, dtype)
    codes, scales = mx.mx_quantize(v, "fp8", scale_group=group)
    return dict(h=h, v=v, codes=codes, scales=scales)


def weight_values(rcodes, rscales) -> np.ndarray:
    """Q4(R) as fp64 [Co][Ci]."""
    return mx.mx_dequantize(mx.unpack_fp4(rcodes), rscales, "fp4")


def product(x64, rcodes, rscales, l1_bits, l2_bits):
    """y = x Q4(R) + (x L1) L2 (F3) in fp64, and the sums of the terms'
    magnitudes that error bounds go by: (y, |x| |Q4(R)|, |x| |L1| |L2|)."""
    x64 = np.asarray(x64, dtype=np.float64)
    w = weight_values(rcodes, rscales).T
    y, main = x64 @ w, np.abs(x64) @ np.abs(w)
    low = np.zeros_like(y)
    if l1_bits is not None and l1_bits.shape[1]:
        l1, l2 = mx.bf16_bits_to_f64(l1_bits), mx.bf16_bits_to_f64(l2_bits)
        y = y + (x64 @ l1) @ l2
        low = (np.abs(x64) @ np.abs(l1)) @ np.abs(l2)
    return y, main, low
