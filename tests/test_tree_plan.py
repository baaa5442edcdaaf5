"""The tree attention's work split on the CPU: every chunk of every item is computed exactly once,
parts of an item land where the merge looks for them, no slot is written twice, and a mask window
is the bits it stands for and reads no word past the request's own.
"""
import ctypes
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("plan") / "tree_plan.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", os.path.join(HERE, "tree_plan_host.cpp"), "-o", so],
                   check=True, capture_output=True)
    L = ctypes.CDLL(so)
    L.plan_per.restype = ctypes.c_longlong
    L.plan_per.argtypes = [ctypes.c_longlong, ctypes.c_int]
    L.plan_cost.argtypes = [ctypes.c_longlong, ctypes.c_int]
    L.plan_head.restype = ctypes.c_longlong
    L.plan_segment.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p]
    L.plan_parts.argtypes = [ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p]
    L.plan_window.restype = ctypes.c_uint
    return L


def request(L, q0, q1, length, T, max_q=256, max_len=1 << 20, gq=4, rows=128):
    out = (ctypes.c_int * 3)()
    ok = L.plan_request(q0, q1, length, T, max_q, max_len, gq, rows, out)
    return bool(ok), out[0], out[1], out[2]


@pytest.mark.parametrize("args,want", [
    ((0, 3, 10, 5), (True, 3, 1, 1)), ((0, 0, 10, 5), (True, 0, 0, 0)), ((0, 64, 129, 64), (True, 64, 2, 2)),
    ((0, 3, 2, 5), (False, 0, 0, 0)), ((-1, 3, 10, 5), (False, 0, 0, 0)), ((3, 2, 10, 5), (False, 0, 0, 0)),
    ((3, 6, 10, 5), (False, 0, 0, 0)), ((0, 257, 300, 999), (False, 0, 0, 0)), ((0, 1, (1 << 20) + 1, 5), (False, 0, 0, 0)),
    ((0, 256, 1 << 20, 256), (True, 256, 8192, 8)),
])
def test_request_counts(lib, args, want):
    assert request(lib, *args) == want


@pytest.mark.parametrize("seed", range(12))
def test_every_chunk_once_and_parts_where_the_merge_looks(lib, seed):
    rng = np.random.default_rng(seed)
    grid = int(rng.choice([1, 2, 7, 152]))
    heads, gq, rows = int(rng.choice([1, 2, 8])), int(rng.choice([1, 4, 7])), int(rng.choice([128, 256]))
    reqs = int(rng.integers(1, 20))
    n = rng.integers(0, 65, reqs)
    lens = n + rng.integers(0, int(rng.choice([50, 3000])), reqs)
    args = [(0, int(k), int(L), 64, 256, 1 << 20, gq, rows) for k, L in zip(n, lens)]
    info = [request(lib, *a) for a in args]
    chunks = sum(heads * g * c for _, _, c, g in info)
    cost = lib.plan_cost(chunks, grid)
    heads_at = []
    for a in args:
        request(lib, *a)
        heads_at.append(heads * lib.plan_head(cost))
    base = np.concatenate([[0], np.cumsum(heads_at)])
    total = int(base[-1])
    per = lib.plan_per(total, grid)
    assert per * grid >= total
    seen, slots, unfinished, load = set(), {}, {}, []
    out = (ctypes.c_longlong * 7)()
    for cta in range(grid):
        pos, end = cta * per, min(total, (cta + 1) * per)
        while pos < end:
            b = int(np.searchsorted(base, pos, side="right")) - 1
            request(lib, *args[b])
            n_chunks, groups = info[b][2:]
            lib.plan_segment(cost, pos - int(base[b]), end - pos, cta, out)
            head, group, c0, c1, part, places, begin = [int(x) for x in out]
            assert 0 <= head < heads and 0 <= group < groups
            assert 0 <= c0 <= c1 <= n_chunks and 0 < places <= end - pos
            pos += places
            if c0 == c1:
                continue
            for c in range(c0, c1):
                assert (b, head, group, c) not in seen
                seen.add((b, head, group, c))
            parts = (ctypes.c_int * 2)()
            lib.plan_parts(group, int(base[b]) + begin, cost, per, parts)
            first, last = parts
            assert first <= cta <= last < grid
            if part < 0:
                assert first == last and (c0, c1) == (0, n_chunks)
            else:
                assert first < last and part not in slots and part == (2 * cta + 1 if cta == first else 2 * cta)
                slots[part] = (b, head, group)
                if c0 == 0:
                    assert cta == first and cta not in unfinished      # one item per CTA for the merge
                    unfinished[cta] = (b, head, group, last)
    assert len(seen) == chunks
    for cta, (b, head, group, last) in unfinished.items():
        for c in range(cta, last + 1):
            assert slots[2 * c + 1 if c == cta else 2 * c] == (b, head, group)
    assert len(slots) == sum(u[3] - cta + 1 for cta, u in unfinished.items())


@pytest.mark.parametrize("seed", range(6))
def test_windows(lib, seed):
    rng = np.random.default_rng(seed)
    for _ in range(300):
        n, ctx = int(rng.integers(1, 257)), int(rng.integers(0, 300))
        words = rng.integers(0, 2 ** 32, -(-n // 32), dtype=np.uint64).astype(np.uint32)
        # the words after the request's own are another row's: planted with ones that must not show
        buf = np.concatenate([words, np.full(2, 0xFFFFFFFF, np.uint32)])
        key = int(rng.integers(0, 18)) * 32
        got = lib.plan_window(buf.ctypes.data_as(ctypes.c_void_p), key, ctx, n)
        for i in range(32):
            k = key + i
            want = k < ctx or (k - ctx < n and (int(words[(k - ctx) // 32]) >> ((k - ctx) % 32)) & 1)
            assert (got >> i) & 1 == int(want), (n, ctx, key, i)
