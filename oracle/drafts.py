"""Drafted token trees on the paged cache, and pages moved inside it (test infrastructure only).

* ``tree_sees``: which drafted tokens of a request each of them sees: its ancestors and
  itself, from the parents' indices (-1: a child of the last cached token).
* ``tree_attention``: a drafted token attends to the ctx cached positions of its request
  and to the drafted positions its row of ``sees`` names; nothing visible gives 0.
  Invisible entries are not touched at all.
* ``copy_blocks``: block dst = block src of the caches, pair by pair.
* ``compact``: the accepted drafted tokens (rising indices) move to the positions after
  the cached ones, from the pages of one block table to those of another.
"""
from __future__ import annotations

import numpy as np

from .attention import _as_f64, first_kv_head, kv_head_of, softmax_rows
from .kv_cache import slot_of
from .tp_block import gqa_partition


def tree_sees(parents) -> np.ndarray:
    """[n, n] boolean: token i sees token j."""
    n = len(parents)
    sees = np.zeros((n, n), dtype=bool)
    for i, p in enumerate(parents):
        if not -1 <= p < i:
            raise ValueError("a parent comes before its child")
        if p >= 0:
            sees[i] = sees[p]
        sees[i, i] = True
    return sees


def mask_words(sees: np.ndarray, words: int) -> np.ndarray:
    """[n, words] int32: bit j % 32 of word j / 32 is sees[:, j]."""
    out = np.zeros((sees.shape[0], words), dtype=np.uint32)
    for i, j in zip(*np.nonzero(sees)):
        out[i, j // 32] |= np.uint32(1 << (int(j) % 32))
    return out.view(np.int32)


def tree_attention(qkv, query_start_loc, seq_lens, block_tables, sees, cache_k, cache_v, nq: int, nkv: int, hd: int,
                   t: int, block_size: int) -> np.ndarray:
    """[t, T, q_per * hd] float64; sees: per request [n, n] boolean. Rows of no request stay 0."""
    a, ck, cv = _as_f64(qkv), _as_f64(cache_k), _as_f64(cache_v)
    q_per, _, _ = gqa_partition(nq, nkv, t)
    out = np.zeros((t, a.shape[1], q_per * hd))
    for b in range(len(seq_lens)):
        q0, n = int(query_start_loc[b]), int(query_start_loc[b + 1]) - int(query_start_loc[b])
        ctx = int(seq_lens[b]) - n
        slots = np.array([slot_of(block_tables, b, j, block_size) for j in range(ctx + n)], dtype=np.int64)
        for i in range(n):
            vis = np.concatenate([np.arange(ctx), ctx + np.nonzero(np.asarray(sees[b])[i, :n])[0]])
            if vis.size == 0:
                continue
            blk, off = slots[vis] // block_size, slots[vis] % block_size
            for r in range(t):
                base = first_kv_head(r, nq, nkv, t)
                for h in range(q_per):
                    g = kv_head_of(r * q_per + h, nq, nkv) - base
                    q = a[r, q0 + i, h * hd:(h + 1) * hd]
                    w = softmax_rows((ck[r, blk, off, g] @ q)[None, :] / np.sqrt(hd))[0]
                    out[r, q0 + i, h * hd:(h + 1) * hd] = w @ cv[r, blk, off, g]
    return out


def copy_blocks(cache: np.ndarray, pairs) -> np.ndarray:
    """cache [t, blocks, ...] after block dst = block src for every pair (src < 0: skipped)."""
    out = cache.copy()
    for s, d in pairs:
        if s >= 0:
            out[:, d] = cache[:, s]
    return out


def compact(cache: np.ndarray, ctx, accepted, src_tables, dst_tables, block_size: int) -> np.ndarray:
    """cache [t, blocks, block_size, ...] after every request's accepted drafts moved together."""
    out = cache.copy()
    for b, kept in enumerate(accepted):
        for j, i in enumerate(kept):
            s, d = slot_of(src_tables, b, ctx[b] + i, block_size), slot_of(dst_tables, b, ctx[b] + j, block_size)
            out[:, d // block_size, d % block_size] = cache[:, s // block_size, s % block_size]
    return out
