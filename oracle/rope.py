"""Rotary positions (oracle; test infrastructure only), float64.

The pages attend keys and queries as a model hands them over, already turned by their
positions (VeloxQuant-MLX page, "Installing and Using It"; FoveatedKV page: 7B GQA shapes of
models with rotary positions).  Pair j of the rotated part of a head at position p is turned
by p * w_j, w_j = base^(-2j / rot), with the usual scalings for longer contexts:

  linear    w_j / factor (positions interpolated);
  base      base * factor^(rot / (rot - 2)) in base's place (rot = 2: unchanged);
  by_parts  w_j (g + (1 - g) / factor), g = clip((context w_j / 2 pi - low) / (high - low)).
"""
from __future__ import annotations

import math

import numpy as np

HALF, INTERLEAVED = "half", "interleaved"


def frequencies(base: float, rot: int, kind: str = "none", factor: float = 1.0, context: float = 0.0,
                low: float = 0.0, high: float = 1.0) -> np.ndarray:
    """Radians per token of each of the rot / 2 pairs."""
    if kind == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    w = np.array([base ** (-2.0 * j / rot) for j in range(rot // 2)], dtype=np.float64)
    if kind == "linear":
        return w / factor
    if kind == "by_parts":
        out = []
        for x in w:
            g = (context * x / (2 * math.pi) - low) / (high - low)
            g = min(1.0, max(0.0, g))
            out.append(x * (g + (1 - g) / factor))
        return np.array(out)
    return w


def pair_index(rot: int, layout: str):
    """Element indices (first, second) of every pair."""
    j = np.arange(rot // 2)
    return (j, j + rot // 2) if layout == HALF else (2 * j, 2 * j + 1)


def apply(x: np.ndarray, positions: np.ndarray, w: np.ndarray, layout: str, scale: float = 1.0,
          transpose: bool = False) -> np.ndarray:
    """x [T, H, d] turned by positions [T]; the transpose turns the other way.  The angle is
    reduced modulo a turn as integers times a fraction would be, in float64 (positions times
    frequencies of test size lose nothing that matters)."""
    y = np.asarray(x, dtype=np.float64).copy()
    rot = 2 * len(w)
    a_at, b_at = pair_index(rot, layout)
    theta = np.asarray(positions, dtype=np.float64)[:, None] * w[None, :]
    c, s = scale * np.cos(theta)[:, None, :], scale * np.sin(theta)[:, None, :]
    if transpose:
        s = -s
    a, b = y[..., a_at].copy(), y[..., b_at].copy()
    y[..., a_at] = a * c - b * s
    y[..., b_at] = b * c + a * s
    return y
