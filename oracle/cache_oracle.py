"""Plain CPU oracle of the 4-bit paged cache and of the head norms with rotation
(numpy, float64), beside the attention oracle and under its rules: test
infrastructure only, no code shared with the CUDA library.

The row format (160 bytes: K codes, V codes, K scales, K minima, V scales, V
minima) and the quantisation are those the public header states.
"""
from __future__ import annotations

import numpy as np

__all__ = ["bf16_toward", "q4_quantise", "q4_values", "q4_pack", "q4_unpack", "norm_rope"]

_GROUP = 32


def bf16_toward(x, up: bool) -> np.ndarray:
    """The nearest bfloat16 number that is not below (up) or not above x."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(x)
    quantum = np.ldexp(1.0, np.maximum(e - 8, -133))  # 8 significant bits; subnormals below 2^-126
    return (np.ceil(x / quantum) if up else np.floor(x / quantum)) * quantum


def q4_quantise(x):
    """Codes int [..., 128], scales and minima [..., 4] of finite rows x [..., 128]."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(*x.shape[:-1], 4, _GROUP)
    m = bf16_toward(g.min(-1), False)
    s = bf16_toward((g.max(-1) - m) / 15.0, True)
    step = np.where(s > 0, s, 1.0)[..., None]
    n = np.rint((g - m[..., None]) / step)  # numpy's rint rounds half to even
    n = np.where(s[..., None] > 0, n, 0.0)
    return n.astype(np.int64).reshape(x.shape), s, m


def q4_values(n, s, m) -> np.ndarray:
    g = np.asarray(n).reshape(*np.shape(n)[:-1], 4, _GROUP)
    return (m[..., None] + s[..., None] * g).reshape(np.shape(n))


def _k_nibble(c: int) -> int:
    return 8 * (4 * ((c >> 3) & 3) + (c >> 5)) + (c & 7)


def _v_nibble(c: int) -> int:
    return 8 * (2 * ((c >> 2) & 7) + (c >> 6)) + 4 * ((c >> 5) & 1) + (c & 3)


def _bf16_bits(x) -> np.ndarray:
    """Bits of numbers that are bfloat16 values already."""
    return (np.asarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)


def q4_pack(k, v) -> np.ndarray:
    """Cache rows uint8 [..., 160] of finite keys and values [..., 128]."""
    lead = np.shape(k)[:-1]
    row = np.zeros((*lead, 160), dtype=np.uint8)
    tail = np.zeros((*lead, 16), dtype=np.uint16)
    for i, (x, place) in enumerate(((k, _k_nibble), (v, _v_nibble))):
        n, s, m = q4_quantise(x)
        for c in range(128):
            p = place(c)
            row[..., 64 * i + (p >> 1)] |= (n[..., c] << (4 * (p & 1))).astype(np.uint8)
        tail[..., 8 * i: 8 * i + 4] = _bf16_bits(s)
        tail[..., 8 * i + 4: 8 * i + 8] = _bf16_bits(m)
    row[..., 128:] = tail.view(np.uint8).reshape(*lead, 32)
    return row


def q4_unpack(row):
    """(codes, scales, minima) of K and of V of cache rows uint8 [..., 160]."""
    row = np.ascontiguousarray(row)
    lead = row.shape[:-1]
    tail = np.ascontiguousarray(row[..., 128:]).view(np.uint16).astype(np.uint32) << 16
    tail = tail.view(np.float32).astype(np.float64).reshape(*lead, 4, 4)
    out = []
    for i, place in enumerate((_k_nibble, _v_nibble)):
        n = np.zeros((*lead, 128), dtype=np.int64)
        for c in range(128):
            p = place(c)
            n[..., c] = (row[..., 64 * i + (p >> 1)] >> (4 * (p & 1))) & 15
        out.append((n, tail[..., 2 * i, :], tail[..., 2 * i + 1, :]))
    return out[0], out[1]


def norm_rope(x, pos, inv_freq, weight=None, eps: float = 1e-6, interleaved: bool = False) -> np.ndarray:
    """x [B, N, H, 128] -> [B, H, N, 128]: RMS norm of each head row (none without
    a weight), then the rotation by the angles pos [B, N] * inv_freq [64]."""
    y = np.asarray(x, dtype=np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    a = np.asarray(pos, dtype=np.float64)[..., None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(a)[:, :, None], np.sin(a)[:, :, None]
    out = np.empty_like(y)
    i, j = (slice(0, None, 2), slice(1, None, 2)) if interleaved else (slice(0, 64), slice(64, 128))
    out[..., i] = y[..., i] * c - y[..., j] * s
    out[..., j] = y[..., j] * c + y[..., i] * s
    return out.transpose(0, 2, 1, 3)
