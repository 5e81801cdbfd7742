"""The layers around the W4A4 ones: row codes, RMS norm, the FP8 linear layer
and cross attention, in plain numpy.

Row codes follow the E4M3 quantiser of ``oracle.attention`` row by row (fp32
steps, byte for byte); everything else is in 64 bits.
"""
from __future__ import annotations

import numpy as np

from . import attention as oatt


def quantize_rows(x):
    """(codes uint8 [rows, cols], scales fp32 [rows]) of a float32 matrix."""
    rows = [oatt.fp8_quantize(r[None, :]) for r in np.asarray(x, np.float32)]
    return np.concatenate([c for c, _ in rows]), np.array([s for _, s in rows], np.float32)


def decode(codes):
    """E4M3 bytes as float64."""
    return np.asarray(oatt.fp8_dequantize(codes, np.float32(1.0)), np.float64)


def rms_norm(x, r=None, w=None, eps=1e-6):
    """(h, y) in float64: h = x + r, y = h / sqrt(mean(h^2) + eps) * w."""
    h = np.asarray(x, np.float64)
    if r is not None:
        h = h + np.asarray(r, np.float64)
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return h, y if w is None else y * np.asarray(w, np.float64)


def gelu_tanh(y):
    return 0.5 * y * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (y + 0.044715 * y ** 3)))


def linear(a, s_a, w, s_w, bias=None, gelu=False, residual=None):
    """act(diag(s_a) a w^T diag(s_w) + bias) + residual in float64; a, w decoded codes."""
    y = (a @ w.T) * np.asarray(s_a, np.float64).reshape(-1, 1) * np.asarray(s_w, np.float64)[None, :]
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    if gelu:
        y = gelu_tanh(y)
    return y if residual is None else y + np.asarray(residual, np.float64)


def cross_attention(q, k, v, heads, kv_heads, batch, kv_batch, kv_len=None, key_mask=None, scale=None):
    """(o, a) in float64, both [batch*Sq, heads*d]: the attention, and the
    same average over |v| (what the rounding of the weights scales with)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    d, sq, sk = q.shape[1] // heads, q.shape[0] // batch, k.shape[0] // kv_batch
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    o, a = np.zeros_like(q), np.zeros_like(q)
    for b in range(batch):
        kb = b if kv_batch > 1 else 0
        on = np.ones(sk, bool)
        if kv_len is not None:
            on &= np.arange(sk) < kv_len[kb]
        if key_mask is not None:
            on &= np.asarray(key_mask[kb], bool)
        if not on.any():
            continue
        for h in range(heads):
            g = h // (heads // kv_heads)
            kk = k[kb * sk:(kb + 1) * sk, g * d:(g + 1) * d][on]
            vv = v[kb * sk:(kb + 1) * sk, g * d:(g + 1) * d][on]
            s = scale * (q[b * sq:(b + 1) * sq, h * d:(h + 1) * d] @ kk.T)
            p = np.exp(s - s.max(axis=1, keepdims=True))
            p /= p.sum(axis=1, keepdims=True)
            o[b * sq:(b + 1) * sq, h * d:(h + 1) * d] = p @ vv
            a[b * sq:(b + 1) * sq, h * d:(h + 1) * d] = p @ np.abs(vv)
    return o, a
