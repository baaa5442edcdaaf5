"""A paged KV cache in 8 bits, and attention of chunks of new tokens with a window (test infrastructure only).

* ``quantise``: head rows as e4m3 values and scale bytes. e4m3 is the 8-bit format with 4 exponent bits (bias 7),
  3 mantissa bits and no infinity: 448 is its largest value, 2^-9 its smallest. Row x gets the smallest integer
  e in [-100, 118] with max|x| <= 448 * 2^e; its codes are the nearest values to x * 2^-e (ties to even, at most
  448 in size), its scale byte is e + 127. A row that is not finite: byte 255, codes 0.
* ``values``: what codes and bytes stand for, code * 2^(byte - 127); NaN rows for 255.
* ``chunk_attention``: a new token at position p of its request attends to positions j <= p with window = 0,
  j > p - window or j < sinks, over the paged cache. Invisible entries are not touched at all.
"""
from __future__ import annotations

import numpy as np

from .attention import _as_f64, first_kv_head, kv_head_of
from .kv_cache import slot_of
from .tp_block import gqa_partition

E_LO, E_HI = -100, 118


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes, from the format's bits (NaN for 0x7f and 0xff)."""
    out = np.empty(256)
    for c in range(256):
        sign, e, m = -1.0 if c & 128 else 1.0, (c >> 3) & 15, c & 7
        out[c] = sign * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        if c & 127 == 127:
            out[c] = np.nan
    return out


def round_e4m3(y: np.ndarray) -> np.ndarray:
    """The nearest e4m3 values, ties to the even code, by search among all of them."""
    mags = e4m3_values()[:127]
    a = np.minimum(np.abs(y), 448.0)
    hi = np.clip(np.searchsorted(mags, a), 1, 126)          # mags[hi - 1] < a <= mags[hi] (or a = 0)
    lo = hi - 1
    below, above = a - mags[lo], mags[hi] - a
    pick = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return np.copysign(mags[pick], y)


def quantise(rows):
    """rows [..., 128] -> (values of the codes float64 [..., 128], scale bytes int [...])."""
    x = _as_f64(rows)
    finite = np.isfinite(x).all(-1)
    top = np.where(finite, np.abs(np.where(np.isfinite(x), x, 0.0)).max(-1), 0.0)
    e = np.full(top.shape, E_LO)
    while True:
        small = (top > 448.0 * np.ldexp(1.0, e)) & (e < E_HI)
        if not small.any():
            break
        e = e + small
    y = round_e4m3(np.where(finite[..., None], np.ldexp(np.where(np.isfinite(x), x, 0.0), -e[..., None]), 0.0))
    return y, np.where(finite, e + 127, 255)


def values(codes, scales):
    """What the values of codes [..., 128] and scale bytes [...] stand for."""
    s = np.asarray(scales, dtype=np.int64)
    out = np.ldexp(_as_f64(codes), (s - 127)[..., None])
    out[s == 255] = np.nan
    return out


def sees(pos: int, length: int, window: int, sinks: int) -> np.ndarray:
    """Boolean [length]: the positions that the token at position pos sees."""
    j = np.arange(length)
    seen = j <= pos
    if window > 0:
        seen &= (j > pos - window) | (j < sinks)
    return seen


def chunk_attention(qkv, query_start_loc, seq_lens, block_tables, cache_k, cache_v, nq: int, nkv: int, hd: int, t: int,
                    block_size: int, window: int = 0, sinks: int = 0, bound: bool = False):
    """[t, T, q_per * hd] float64; rows of no request stay 0. With bound (for tolerances): also sum p |v| and
    sqrt(sum p^2 v^2) of every element, and the largest sum |q_i k_i| / sqrt(hd) of every row's scores."""
    a, ck, cv = _as_f64(qkv), _as_f64(cache_k), _as_f64(cache_v)
    q_per, _, _ = gqa_partition(nq, nkv, t)
    out = np.zeros((t, a.shape[1], q_per * hd))
    size, spread, score = np.zeros_like(out), np.zeros_like(out), np.zeros((t, a.shape[1], q_per))
    for b in range(len(seq_lens)):
        q0, n, L = int(query_start_loc[b]), int(query_start_loc[b + 1]) - int(query_start_loc[b]), int(seq_lens[b])
        if n == 0:
            continue
        see = np.stack([sees(L - n + i, L, window, sinks) for i in range(n)])
        need = see.any(0)                                    # what no token sees is not touched
        slots = np.array([slot_of(block_tables, b, j, block_size) for j in np.nonzero(need)[0]], dtype=np.int64)
        blk, off, see = slots // block_size, slots % block_size, see[:, need]
        for r in range(t):
            base = first_kv_head(r, nq, nkv, t)
            for h in range(q_per):
                g = kv_head_of(r * q_per + h, nq, nkv) - base
                q, k, v = a[r, q0:q0 + n, h * hd:(h + 1) * hd], ck[r, blk, off, g], cv[r, blk, off, g]
                with np.errstate(invalid="ignore"):
                    s = np.where(see, q @ k.T / np.sqrt(hd), -np.inf)
                    w = np.exp(s - s.max(-1, keepdims=True))
                    w /= w.sum(-1, keepdims=True)
                    clean = np.isfinite(v).all(-1)
                    o = w[:, clean] @ v[clean]
                    for j in np.nonzero(~clean)[0]:         # a value that is not finite reaches those that see it alone
                        o[see[:, j]] += w[see[:, j], j, None] * v[j]
                out[r, q0:q0 + n, h * hd:(h + 1) * hd] = o
                if bound:
                    size[r, q0:q0 + n, h * hd:(h + 1) * hd] = w @ np.abs(v)
                    spread[r, q0:q0 + n, h * hd:(h + 1) * hd] = np.sqrt(w ** 2 @ v ** 2)
                    score[r, q0:q0 + n, h] = np.where(see, np.abs(q) @ np.abs(k).T / np.sqrt(hd), 0).max(-1)
    return (out, size, spread, score) if bound else out
