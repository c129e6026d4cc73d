"""Reference definitions, in fp64 NumPy, of the operators that keep a paged
KV cache within a budget: rotary positions, the attention weight paid to each
cached token, the positions a budget keeps, and the compaction of their rows.

TEST INFRASTRUCTURE.  Only ``tests/`` may import this module; the library
never calls it and shares no code with it.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["rope", "scores_update", "select", "compact_head"]


def rope(x: np.ndarray, positions: np.ndarray, inv_freq: np.ndarray, interleaved: bool = False,
         amplitude: float = 1.0) -> np.ndarray:
    """x [T, H, D] (any float type) rotated to positions [T], in fp64: pair i
    of a head turns by positions * inv_freq[i]; the rest is copied."""
    y = x.astype(np.float64).copy()
    r = len(inv_freq)
    for t in range(x.shape[0]):
        for i in range(r):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
            turns = math.fmod(int(positions[t]) * float(inv_freq[i]), 2 * math.pi)
            c, s = amplitude * math.cos(turns), amplitude * math.sin(turns)
            x1, x2 = x[t, :, a].astype(np.float64), x[t, :, b].astype(np.float64)
            y[t, :, a] = x1 * c - x2 * s
            y[t, :, b] = x2 * c + x1 * s
    return y


def scores_update(q: np.ndarray, K: np.ndarray, old: np.ndarray, scale: float, causal: bool = True,
                  decay: float = 1.0) -> np.ndarray:
    """One sequence's scores [Hkv, L] after a step: q [n, Hq, D] its queries,
    K [L, Hkv, D] its cached keys, old [Hkv, L] the scores before."""
    n, Hq, _ = q.shape
    L, Hkv, _ = K.shape
    G = Hq // Hkv
    out = np.zeros((Hkv, L))
    for i in range(n):
        seen = L - n + i + 1 if causal else L
        for h in range(Hq):
            z = scale * (K[:seen, h // G].astype(np.float64) @ q[i, h].astype(np.float64))
            w = np.exp(z - z.max())
            out[h // G, :seen] += w / w.sum()
    if decay != 0.0 and n > 0:
        out[:, :L - n] += decay * old[:, :L - n].astype(np.float64)
    return out if n > 0 else old.astype(np.float64)


def select(scores: np.ndarray, L: int, budget: int, sink: int = 0, recent: int = 0) -> list[int]:
    """Kept positions of one (sequence, head), ascending."""
    if L <= budget:
        return list(range(L))
    middle = range(sink, L - recent)
    worth = lambda j: -math.inf if math.isnan(scores[j]) else float(scores[j])  # noqa: E731
    # a NaN below -inf, then by value, then the lower position
    best = sorted(middle, key=lambda j: (math.isnan(scores[j]), -worth(j), j))[:budget - sink - recent]
    return sorted(list(range(sink)) + best + list(range(L - recent, L)))


def compact_head(pool: np.ndarray, src_table, dst_table, kept, head: int, source: np.ndarray | None = None) -> None:
    """Moves one head's kept rows in place: pool [NB, bs, Hkv, D] of any
    type; `source` (default: a copy of pool) holds the rows as they were."""
    bs = pool.shape[1]
    src = pool.copy() if source is None else source
    for r, j in enumerate(kept):
        pool[dst_table[r // bs], r % bs, head] = src[src_table[j // bs], j % bs, head]
