"""Attention of chunks of new tokens over the compressed cache, and of windows with sinks (oracle;
test infrastructure only).

A sequence's tokens are those of its tiers, one tier after the other; its chunk is the last of
them.  Query i of T stands at p = L - T + i and attends, as in ``attention.attend`` (float64), to the
positions t <= p that lie in its window (t > p - window; window 0: all) or among the first
``sinks``.  A query that sees nothing gives zeros.
"""
from __future__ import annotations

from typing import Sequence

import numpy as np

from . import attention


def sees(p: int, length: int, window: int = 0, sinks: int = 0) -> np.ndarray:
    """Which of the positions 0 .. length - 1 a query at position p sees."""
    t = np.arange(length)
    return (t <= p) & ((t > p - window) | (t < sinks) | (window == 0))


def chunk_attention(q16: np.ndarray, tiers: Sequence[attention.TierState], offsets: Sequence[int], window: int = 0,
                    sinks: int = 0) -> np.ndarray:
    """q16 [T, Hq, d] (fp16); sequence b's queries are offsets[b] .. offsets[b + 1] - 1.  Returns
    float64 [T, Hq, d]; rows of no chunk are zero."""
    hkv = tiers[0].k.signs.shape[0]
    grp = q16.shape[1] // hkv
    out = np.zeros(q16.shape, dtype=np.float64)
    for b in range(len(offsets) - 1):
        count = offsets[b + 1] - offsets[b]
        length = sum(int(t.lens[b]) for t in tiers)
        for g in range(hkv):
            keys, values = attention.dequantised_kv(tiers, b, g)
            for i in range(count):
                seen = sees(length - count + i, length, window, sinks)
                if not seen.any():
                    continue
                for h in range(g * grp, (g + 1) * grp):
                    q = q16[offsets[b] + i, h].astype(np.float64)
                    extra = attention.sketch_terms(tiers, b, g, q)[seen]
                    out[offsets[b] + i, h] = attention.attend(q, keys[seen], values[seen], extra)
    return out
