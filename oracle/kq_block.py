"""Float64 oracle of the operators around a W4A4 layer: the MXFP4 K/V cache,
the attention over it and the product's epilogue.

Plain numpy from the definitions; the E2M1 and E8M0 rules come from
``kq_oracle`` (blocks of 32, the floor rule, ties to the even code).
"""
from __future__ import annotations

import math

import numpy as np

from . import kq_oracle as o


# ------------------------------------------------------------------- cache
def quantize_rows(x):
    """Codes [..., Dp/2] and scale bytes [..., Dp/32] of rows [..., D] (the
    last block padded with zeros)."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    dp = -(-d // 32) * 32
    rows = np.zeros(x.shape[:-1] + (dp,))
    rows[..., :d] = x
    codes, s = o.mxfp4_quantize(rows.reshape(-1, dp))
    q = o.pack_codes(codes)
    return q.reshape(x.shape[:-1] + (dp // 2,)), s.reshape(x.shape[:-1] + (dp // 32,))


def decode_rows(codes, scales, d):
    dp = 2 * codes.shape[-1]
    y = o.dequantize(codes.reshape(-1, dp // 2), scales.reshape(-1, dp // 32))
    return y.reshape(codes.shape[:-1] + (dp,))[..., :d]


def place(table, page_size, pages, b, pos):
    """(page, slot) of a position, or None where it has no page in the pool."""
    if pos < 0 or pos // page_size >= table.shape[1]:
        return None
    page = int(table[b, pos // page_size])
    return (page, pos % page_size) if 0 <= page < pages else None


def cache_write(codes, scales, table, x, start, lens):
    """Rows x [B, T, H, D] into codes / scales [pages, H, page_size, .], in
    place; returns how many rows had no page."""
    q, s = quantize_rows(x)
    lost = 0
    for b in range(x.shape[0]):
        for t in range(min(int(lens[b]), x.shape[1])):
            at = place(table, codes.shape[2], codes.shape[0], b, int(start[b]) + t)
            if at is None:
                lost += 1
                continue
            codes[at[0], :, at[1]] = q[b, t]
            scales[at[0], :, at[1]] = s[b, t]
    return lost


def cache_read(codes, scales, table, lens, tokens, start, d):
    y = np.zeros((table.shape[0], tokens, codes.shape[1], d))
    for b in range(table.shape[0]):
        for t in range(min(int(lens[b]), tokens)):
            at = place(table, codes.shape[2], codes.shape[0], b, int(start[b]) + t)
            if at is not None:
                y[b, t] = decode_rows(codes[at[0], :, at[1]], scales[at[0], :, at[1]], d)
    return y


# --------------------------------------------------------------- attention
def attention(q, k, v, lens, causal=False, scale=None, seen=None):
    """q [B, M, H, D], k and v [B, L, Hkv, D]; returns (out, lse [B, H, M],
    terms, logit) with terms = sum_p softmax_p |V[p]| and logit [B, H, M] the
    largest scale * sum |q| |k| of a seen position: the magnitudes of what the
    two products add up.  seen: optional [B, L] positions that count."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    B, M, H, D = q.shape
    L, Hkv = k.shape[1], k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    out, terms = np.zeros(q.shape), np.zeros(q.shape)
    lse, logit = np.full((B, H, M), -np.inf), np.zeros((B, H, M))
    for b in range(B):
        n = max(0, min(int(lens[b]), L))
        for h in range(H):
            kh, vh = k[b, :n, h // (H // Hkv)], v[b, :n, h // (H // Hkv)]
            for m in range(M):
                ok = np.arange(n) <= n - M + m if causal else np.ones(n, dtype=bool)
                if seen is not None:
                    ok = ok & seen[b, :n]
                if not ok.any():
                    continue
                s = scale * (kh[ok] @ q[b, m, h])
                w = np.exp(s - s.max())
                lse[b, h, m] = s.max() + math.log(w.sum())
                w = w / w.sum()
                out[b, m, h] = w @ vh[ok]
                terms[b, m, h] = w @ np.abs(vh[ok])
                logit[b, h, m] = abs(scale) * (np.abs(kh[ok]) @ np.abs(q[b, m, h])).max()
    return out, lse, terms, logit


# ---------------------------------------------------------------- epilogue
def activation(x, name):
    if name == "none":
        return x
    if name == "gelu_tanh":
        return 0.5 * x * (1 + np.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))
    if name == "gelu":
        return 0.5 * x * np.vectorize(math.erfc, otypes=[np.float64])(-x / math.sqrt(2))
    if name == "silu":
        with np.errstate(over="ignore"):
            return x / (1 + np.exp(-x))
    raise ValueError(name)


def epilogue(y, bias=None, act="none", gate=None, tokens=1, residual=None):
    """residual + gate[row // tokens] * act(y + bias), each part optional."""
    y = np.asarray(y, dtype=np.float64)
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)
    y = activation(y, act)
    if gate is not None:
        y = y * np.asarray(gate, dtype=np.float64)[np.arange(y.shape[0]) // tokens]
    return y if residual is None else y + np.asarray(residual, dtype=np.float64)
