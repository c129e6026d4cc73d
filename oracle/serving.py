"""Reference definitions, in fp64 NumPy, of attention with a sliding window and
sinks, of the RMS norm of q and k heads before their rotation, and of pools of
8-bit codes with a scale for each block and kv head.

TEST INFRASTRUCTURE.  Only ``tests/`` and ``__graft_entry__.smoke()`` may import
this module; the library never calls it and shares no code with it.
"""
from __future__ import annotations

import math

import numpy as np

from oracle import fp8

__all__ = ["window_attend", "head_norm", "block_scale", "write_blocks", "block_values"]


def window_attend(q, K, V, scale: float, window: int = 0, num_sink: int = 0, causal: bool = True) -> np.ndarray:
    """One sequence: q [n, Hq, D], K and V [L, Hkv, D] in fp64.  The query at
    position p = L - n + i sees the keys j <= p (all of them when not causal)
    and, with a window, of these those with j > p - window or j < num_sink.
    Hidden keys have no part in it, whatever they hold."""
    n, Hq, D = q.shape
    L, Hkv, _ = K.shape
    out = np.zeros((n, Hq, D))
    for i in range(n):
        p = L - n + i
        seen = [j for j in range(p + 1 if causal else L) if not window or j > p - window or j < num_sink]
        for h in range(Hq):
            g = h // (Hq // Hkv)
            z = scale * (K[seen, g] @ q[i, h])
            w = np.exp(z - z.max())
            out[i, h] = (w / w.sum()) @ V[seen, g]
    return out


def head_norm(x: np.ndarray, weight, eps: float) -> np.ndarray:
    """x [T, H, D]: each head over its root mean square, times weight [D] (None: 1)."""
    x = x.astype(np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y if weight is None else y * np.asarray(weight, dtype=np.float64)


def block_scale(top: float) -> float:
    """The least power of two in [2^-60, 2^60] whose 448-fold reaches ``top``."""
    if not top > 0.0:
        return 2.0 ** -60
    e = -60
    while e < 60 and 448.0 * 2.0 ** e < top:
        e += 1
    return 2.0 ** e


def write_blocks(rows: np.ndarray, slots, codes: np.ndarray, scales: np.ndarray) -> None:
    """In place: rows [T, Hkv, D] (fp32 values) into codes [NB, bs, Hkv, D]
    (uint8) and scales [NB, Hkv] at ``slots`` (< 0 skips)."""
    bs = codes.shape[1]
    slots = np.asarray(slots)
    for b in sorted({int(s) // bs for s in slots if s >= 0}):
        mine = [t for t, s in enumerate(slots) if s >= 0 and int(s) // bs == b]
        begins = any(int(slots[t]) % bs == 0 for t in mine)
        for h in range(codes.shape[2]):
            top = np.abs(rows[mine, h]).astype(np.float64)
            top = float(np.nanmax(np.where(np.isnan(top), 0.0, top)))
            scale = block_scale(top)
            if not begins:
                old = float(scales[b, h])
                if old >= scale:
                    scale = old
                else:
                    codes[b, :, h] = fp8.e4m3_encode((fp8.dequantize(codes[b, :, h], 1.0) * (old / scale)).astype(np.float32))
            scales[b, h] = scale
            for t in mine:
                codes[b, int(slots[t]) % bs, h] = fp8.e4m3_encode((rows[t, h].astype(np.float64) / scale).astype(np.float32))


def block_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The pool's values in fp64."""
    return fp8.dequantize(codes, 1.0) * scales.astype(np.float64)[:, None, :, None]
