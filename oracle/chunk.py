"""Attention of a chunk of new tokens, and rotary positions, in fp64.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The query of the chunk's token i, with N tokens held before the chunk, sees
what a decode step sees once the chunk's tokens 0..i are appended: it is
``attention.decode_head`` over the first N + i + 1 tokens.
"""
from __future__ import annotations

import math

import numpy as np

from .attention import decode_head
from .quant import code_value, dequantize_per_token, middle_blocks


def chunk_head(q, K, V, policy: int, kept, N: int, S: int, W: int, W_loc: int, special_flags=None) -> np.ndarray:
    """q [n, G, d]: the chunk's queries of the heads that share one KV head;
    K, V [N + n, d]: its dense history, the chunk's tokens last.  [n, G, d]."""
    return np.stack([decode_head(q[i], K, V, policy, kept, N + i + 1, S, W, W_loc, special_flags)
                     for i in range(len(q))])


def sealed_keys(codes, scales, fmt: str = "int8") -> np.ndarray:
    """The keys of a sealed block [128, k] as chunk attention takes them: the block's
    scales moved by a power of two so that the largest lies in [2^6, 2^7), each
    rounded to f16, and their products with the codes rounded to f16."""
    s = np.asarray(scales, np.float32)
    e = max(int(s.max().view(np.uint32) >> 23) - 127 - 6, -126)
    s16 = (s * np.float32(2.0 ** -e)).astype(np.float16).astype(np.float64)
    return (code_value(codes, fmt) * s16).astype(np.float16).astype(np.float64) * 2.0 ** e


def sealed_history(K, V, kept, policy: int, N: int, S: int, W: int, fmt: str = "int8"):
    """``quant.quantized_history`` with the sealed keys as chunk attention takes
    them."""
    Kq, Vq = np.array(K[:N], dtype=np.float64), np.array(V[:N], dtype=np.float64)
    if policy != 0:
        return Kq, Vq
    kept = np.asarray(kept, dtype=np.int64)
    for j, (kc, ks, vc, vs) in enumerate(middle_blocks(K, V, kept, N, S, W, fmt)):
        rows = np.arange(S + 128 * j, S + 128 * (j + 1))
        Kq[np.ix_(rows, kept)] = sealed_keys(kc, ks, fmt)
        Vq[rows] = dequantize_per_token(vc, vs, fmt)
    return Kq, Vq


def rope_frequencies(dim: int, base: float, scaling: str = "none", factor: float = 1.0, trained: int = 0,
                     low: float = 0.0, high: float = 0.0) -> np.ndarray:
    """Angle per position of each pair, float64 [dim / 2]."""
    i = np.arange(dim // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (dim / (dim - 2))
    w = base ** (-2.0 * i / dim)
    turns = trained * w / (2 * math.pi)
    if scaling == "linear":
        return w / factor
    if scaling == "yarn":
        def at(n):                       # the (real) pair index that turns n times in the trained length
            return dim * math.log(trained / (n * 2 * math.pi)) / (2 * math.log(base))
        first = max(math.floor(at(high or 32.0)), 0)
        last = min(math.ceil(at(low or 1.0)), dim - 1)
        r = np.clip((i - first) / max(last - first, 1e-3), 0.0, 1.0)
        return w * (1 - r) + w / factor * r
    if scaling == "bands":
        low, high = low or 1.0, high or 4.0
        s = np.clip((turns - low) / (high - low), 0.0, 1.0)
        return w * s + w / factor * (1 - s)
    return w


def rope(x, positions, frequencies, layout: str = "half", magnitude: float = 1.0) -> np.ndarray:
    """x [tokens, heads, d] turned by positions [tokens], float64."""
    x = np.array(x, dtype=np.float64)
    half = len(frequencies)
    angle = np.asarray(positions, np.float64)[:, None, None] * frequencies
    c, s = magnitude * np.cos(angle), magnitude * np.sin(angle)
    a, b = (slice(0, half), slice(half, 2 * half)) if layout == "half" else \
        (slice(0, 2 * half, 2), slice(1, 2 * half, 2))
    xa, xb = x[..., a].copy(), x[..., b].copy()
    x[..., a] = xa * c - xb * s
    x[..., b] = xb * c + xa * s
    return x
