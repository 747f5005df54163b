"""Plain float64 definitions of the operators by which a decoder reads the
encoder's states.  Test infrastructure only.

Pins (tests/test_oracle_decoder_reads.py):

  e4m3_codes, quantize_fp8   torch's float8_e4m3fn cast on scaled values; the
                             scale's defining inequality checked directly
  linear_fp8                 float64 product of torch's decoded codes
  cross_attention            torch scaled_dot_product_attention in float64
  cross_attention_weights    rows sum to one, and W V = cross_attention
"""
from __future__ import annotations

import numpy as np

__all__ = ["e4m3_values", "e4m3_codes", "quantize_fp8", "dequantize_fp8", "linear_fp8", "cross_attention",
           "cross_attention_weights"]


def e4m3_values() -> np.ndarray:
    """Value of each e4m3 code 0..255 (4 exponent bits with bias 7, 3 mantissa
    bits, no infinities, S.1111.111 = NaN), from the format's definition."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        mag = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if (c & 127) == 127 else (-mag if c & 128 else mag)
    return out


def e4m3_codes(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 code, ties to the even code, |v| <= 448; NaN and infinities
    give the NaN code of their sign."""
    grid = e4m3_values()[:127]
    a = np.abs(np.asarray(v, np.float64))
    fin = np.where(np.isfinite(a), a, 0.0)
    hi = np.clip(np.searchsorted(grid, fin), 1, 126)
    lo = hi - 1
    dl, dh = fin - grid[lo], grid[hi] - fin
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.isfinite(a), code, 127)
    return (code | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def quantize_fp8(x: np.ndarray, block_rows: int = 1):
    """(codes uint8 [M, K], exponents int [ceil(M / block_rows), ceil(K / 128)]):
    per block the smallest s in [-127, 120] with max |x| <= 448 * 2^s over the
    finite values (0 for a block of zeros), code = e4m3(x 2^-s)."""
    x = np.asarray(x, np.float64)
    M, K = x.shape
    s = np.zeros((-(-M // block_rows), -(-K // 128)), np.int64)
    codes = np.empty((M, K), np.uint8)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            b = x[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128]
            a = np.abs(b[np.isfinite(b)])
            top = a.max() if a.size else 0.0
            if top > 0:
                e = -127
                while top > 448 * 2.0 ** e:
                    e += 1
                s[i, j] = e
            codes[i * block_rows:(i + 1) * block_rows, j * 128:(j + 1) * 128] = e4m3_codes(b * 2.0 ** -s[i, j])
    return codes, s


def dequantize_fp8(codes: np.ndarray, s: np.ndarray, block_rows: int) -> np.ndarray:
    M, K = codes.shape
    scale = np.repeat(np.repeat(2.0 ** s.astype(np.float64), block_rows, 0)[:M], 128, 1)[:, :K]
    return e4m3_values()[codes] * scale


def linear_fp8(xc, xs, wc, ws, bias=None) -> np.ndarray:
    """X W^T + bias on the values that codes and exponents stand for."""
    y = dequantize_fp8(xc, xs, 1) @ dequantize_fp8(wc, ws, 128).T
    return y if bias is None else y + np.asarray(bias, np.float64)


def _softmax(s: np.ndarray) -> np.ndarray:
    p = np.exp(s - s.max(-1, keepdims=True))
    return p / p.sum(-1, keepdims=True)


def cross_attention(q, k, v, cu_q, cu_k) -> np.ndarray:
    """Rows i of segment j attend to the states cu_k[j] .. cu_k[j + 1]:
    softmax(q k^T / 8) v per 64-wide head, head h reading k/v head h / group;
    a segment without states gives zeros ([CW], whisper-small decoder)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    H, group = q.shape[1] // 64, q.shape[1] // k.shape[1]
    out = np.zeros(q.shape)
    for j in range(len(cu_q) - 1):
        qs, ks = slice(cu_q[j], cu_q[j + 1]), slice(cu_k[j], cu_k[j + 1])
        if cu_k[j + 1] <= cu_k[j]:
            continue
        for h in range(H):
            c, g = slice(64 * h, 64 * h + 64), slice(64 * (h // group), 64 * (h // group) + 64)
            out[qs, c] = _softmax(q[qs, c] @ k[ks, g].T / 8) @ v[ks, g]
    return out


def cross_attention_weights(q, k, cu_q, cu_k, heads, width: int) -> np.ndarray:
    """The softmax rows themselves for the listed heads, [len(heads), Tq, width],
    columns past a segment's states zero ([CW], "with cross-attentions")."""
    q, k = (np.asarray(t, np.float64) for t in (q, k))
    group = q.shape[1] // k.shape[1]
    out = np.zeros((len(heads), q.shape[0], width))
    for j in range(len(cu_q) - 1):
        qs, ks = slice(cu_q[j], cu_q[j + 1]), slice(cu_k[j], cu_k[j + 1])
        n = cu_k[j + 1] - cu_k[j]
        if n <= 0:
            continue
        for i, h in enumerate(heads):
            c, g = slice(64 * h, 64 * h + 64), slice(64 * (h // group), 64 * (h // group) + 64)
            out[i, qs, :n] = _softmax(q[qs, c] @ k[ks, g].T / 8)
    return out
