"""Rotary positions and per-head norms of q and k (test infrastructure only).

The pages define no positional rotation; these are the published formulas.

* frequencies: f_i = base^(-2i/d), i < d/2; position interpolation divides them by a
  factor; NTK-aware scaling changes the base; frequency bands leave the fast pairs,
  divide the slow ones and blend between (by turns over the original context); YaRN
  (Peng et al., 2023) ramps between two turn counts and multiplies cos and sin by
  0.1 ln(factor) + 1.
* rotation of a pair (a, b) by angle p f_i: (a c - b s, b c + a s); the pairs are
  (x_i, x_{i+d/2}) ("half") or (x_2i, x_2i+1) ("interleaved"), i < d/2, of the first d
  elements of a head.
* norm: x / sqrt(mean(x^2) + eps) * gamma per head, before the rotation.
"""
from __future__ import annotations

import math

import numpy as np

from .attention import _as_f64
from .tp_block import gqa_partition


def rope_frequencies(d: int, base: float, scaling: str = "none", factor: float = 1.0, original: int = 0,
                     low: float = 1.0, high: float = 4.0, beta_slow: float = 1.0, beta_fast: float = 32.0):
    """(f [d/2], multiplier of cos and sin)."""
    out, m = [], 1.0
    for i in range(d // 2):
        f = base ** (-2.0 * i / d)
        if scaling == "linear":
            f = f / factor
        elif scaling == "ntk":
            f = (base * factor ** (d / (d - 2.0))) ** (-2.0 * i / d)
        elif scaling == "bands":
            wavelength = 2.0 * math.pi / f
            if wavelength > original / low:
                f = f / factor
            elif wavelength >= original / high:
                u = (original / wavelength - low) / (high - low)
                f = (1.0 - u) * f / factor + u * f
        elif scaling == "yarn":
            def pair(turns):
                return d * math.log(original / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))
            lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), d - 1)
            u = min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 0.001)))
            f = f / factor * u + f * (1.0 - u)
            m = 0.1 * math.log(factor) + 1.0 if factor > 1.0 else 1.0
        out.append(f)
    return np.array(out), m


def rotate_pairs(x: np.ndarray, angle: np.ndarray, interleaved: bool, scale: float = 1.0) -> np.ndarray:
    """Rotate the first 2 * angle.shape[-1] elements of the rows of x [n, hd] by angle [n, d/2]."""
    half = angle.shape[-1]
    y = x.copy()
    c, s = np.cos(angle) * scale, np.sin(angle) * scale
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y[:, a] = x[:, a] * c - x[:, b] * s
    y[:, b] = x[:, b] * c + x[:, a] * s
    return y


def head_norm(x: np.ndarray, gamma: np.ndarray, eps: float) -> np.ndarray:
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * gamma


def qk_norm_rope(qkv, positions, inv_freq, nq: int, nkv: int, hd: int, t: int, interleaved: bool = False,
                 scale: float = 1.0, q_gamma=None, k_gamma=None, eps: float = 1e-6) -> np.ndarray:
    """[t, T, w_s] with q and k heads normed (where a gamma is given) and rotated; a token at a
    negative position keeps its row as it is."""
    a = _as_f64(qkv).copy()
    q_per, kv_per, _ = gqa_partition(nq, nkv, t)
    pos = np.asarray(positions, dtype=np.float64)
    live = pos >= 0
    angle = pos[live, None] * np.asarray(inv_freq)[None, :]
    for r in range(t):
        for h in range(q_per + kv_per):
            x = a[r, live, h * hd:(h + 1) * hd]
            gamma = q_gamma if h < q_per else k_gamma
            if gamma is not None:
                x = head_norm(x, _as_f64(gamma), eps)
            a[r, live, h * hd:(h + 1) * hd] = rotate_pairs(x, angle, interleaved, scale)
    return a
