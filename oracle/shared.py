"""Decode attention for groups of sequences on shared prefixes (oracle; test infrastructure).

A sequence's context is its group's prefix followed by its own tokens, all in one softmax
(XQuant page, step 4: softmax(q K^T / sqrt(d)) V over the whole context); sharing the prefix
changes where its pages are found, not the result.
"""
from __future__ import annotations

import dataclasses
from typing import List, Sequence

import numpy as np

from .attention import TierState


def group_of(offsets: Sequence[int], batch: int) -> np.ndarray:
    """The group of every sequence, -1 where it has none: group i is the sequences
    offsets[i] .. offsets[i + 1] - 1."""
    out = np.full(batch, -1, dtype=np.int64)
    for i in range(len(offsets) - 1):
        out[offsets[i]:offsets[i + 1]] = i
    return out


def as_tiers(prefix: Sequence[TierState], offsets: Sequence[int], own: Sequence[TierState], batch: int) -> List[TierState]:
    """The prefix tiers (tables and lengths per group) as tiers of every sequence, then the
    sequences' own."""
    g = group_of(offsets, batch)
    tiers = []
    for t in prefix:
        table = np.asarray(t.block_table)[np.maximum(g, 0)]
        lens = np.where(g >= 0, np.asarray(t.lens)[np.maximum(g, 0)], 0)
        tiers.append(dataclasses.replace(t, block_table=table, lens=lens))
    return tiers + list(own)
