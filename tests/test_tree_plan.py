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
    L.plan_item.restype = ctypes.c_longlong
    L.plan_item.argtypes = [ctypes.c_int]
    L.plan_segment.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p]
    L.plan_parts.argtypes = [ctypes.c_longlong, ctypes.c_int, ctypes.c_longlong, ctypes.c_void_p]
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
    info = [request(lib, 0, int(k), int(L), 64, gq=gq, rows=rows) for k, L in zip(n, lens)]
    base = np.concatenate([[0], np.cumsum([heads * g * lib.plan_item(c) for _, _, c, g in info])])
    chunks = sum(heads * g * c for _, _, c, g in info)
    total = int(base[-1])
    per = lib.plan_per(total, grid)
    assert per * grid >= total
    seen, slots, unfinished = set(), {}, {}
    out = (ctypes.c_longlong * 5)()
    for cta in range(grid):
        pos, end = cta * per, min(total, (cta + 1) * per)
        while pos < end:
            b = int(np.searchsorted(base, pos, side="right")) - 1
            lib.plan_segment(pos - int(base[b]), info[b][2], end - pos, cta, out)
            unit, c0, c1, part, places = [int(x) for x in out]
            assert 0 <= unit < heads * info[b][3] and 0 <= c0 <= c1 <= info[b][2] and 0 < places <= end - pos
            pos += places
            if c0 == c1:
                assert pos == end                          # the range ends before the item's first chunk
                continue
            for c in range(c0, c1):
                assert (b, unit, c) not in seen
                seen.add((b, unit, c))
            parts = (ctypes.c_int * 2)()
            lib.plan_parts(int(base[b]) + unit * lib.plan_item(info[b][2]), info[b][2], per, parts)
            first, last = parts
            assert first <= cta <= last < grid
            if part < 0:
                assert first == last and (c0, c1) == (0, info[b][2])
            else:
                assert first < last and part not in slots and part == (2 * cta + 1 if cta == first else 2 * cta)
                slots[part] = (b, unit)
                if c0 == 0:
                    assert cta == first and cta not in unfinished      # one item per CTA for the merge
                    unfinished[cta] = (b, unit, last)
    assert len(seen) == chunks
    for cta, (b, unit, last) in unfinished.items():
        for c in range(cta, last + 1):
            assert slots[2 * c + 1 if c == cta else 2 * c] == (b, unit)
    assert len(slots) == sum(last - cta + 1 for cta, (_, _, last) in unfinished.items())


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
