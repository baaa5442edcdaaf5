"""The chunk attention's work split on the CPU: which keys an item takes, the places of a request's items in
closed form, and, with the launch's own grid, that every chunk is computed once and the merge reads only slots
that this call wrote for that item."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("chunk") / "chunk_plan.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", os.path.join(HERE, "chunk_plan_host.cpp"), "-o", so],
                   check=True, capture_output=True)
    L = ctypes.CDLL(so)
    L.floor_sum.restype = ctypes.c_longlong
    L.sees.restype = L.item_sees.restype = ctypes.c_uint
    return L


def visible(pos, window, sinks):
    return {j for j in range(pos + 1) if window == 0 or j > pos - window or j < sinks}


def test_floor_sum(lib):
    rng = np.random.default_rng(0)
    for _ in range(500):
        n, a, b = int(rng.integers(0, 200)), int(rng.integers(0, 257)), int(rng.integers(0, 100000))
        m = int(rng.choice([1, 2, 7, 128, 128, 128]))
        assert lib.floor_sum(n, m, a, b) == sum((a * i + b) // m for i in range(n))


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (5, 3), (64, 200), (128, 4), (129, 128), (300, 0), (40, 129)])
def test_visibility_bits(lib, window, sinks):
    for pos in (0, 1, 31, 32, 127, 128, 200, 383, 500):
        see = visible(pos, window, sinks)
        for key in range(0, 512, 32):
            want = sum(1 << i for i in range(32) if key + i in see)
            assert lib.sees(key, pos, window, sinks) == want, (pos, key)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 1), (100, 5), (128, 128), (129, 129), (300, 0), (17, 260), (1000, 1)])
@pytest.mark.parametrize("tokens", [1, 2, 36, 64, 256])
def test_item_goes_through_the_keys_that_its_tokens_see(lib, window, sinks, tokens):
    out = (ctypes.c_int * 8192)()
    for p0 in (0, 1, 100, 127, 128, 255, 300, 511, 640, 1000):
        p1 = p0 + tokens - 1
        got = list(out[:lib.item_keys(p0, p1, window, sinks, out)])
        see = {p: visible(p, window, sinks) for p in {p0, (p0 + p1) // 2, p1}}
        need = set().union(*see.values()) | set(range(p0, p1 + 1))
        # every key once, in order, 16 on end at a time; none of a chunk without need
        assert got == sorted(set(got)) and need <= set(got)
        assert all(got[i + 15] == got[i] + 15 and got[i] % 16 == 0 for i in range(0, len(got), 16))
        lo = max(p0 - window + 1, 0) if window else 0
        listed = {j for j in range(p1 + 1) if j >= lo // 16 * 16 or j < -(-sinks // 16) * 16}
        assert len(got) == -(-len(listed) // 128) * 128 or set(got) == set(range(len(got)))
        for x in range(0, len(got), 16):
            for p in see:
                want = sum(1 << i for i in range(min(32, len(got) - x)) if got[x + i] in see[p])
                bits = lib.item_sees(p0, p1, window, sinks, x, p) & ((1 << min(32, len(got) - x)) - 1)
                assert bits == want, (p0, p, x)
        # keys that are not masked are seen by all
        for n in (64, 128):
            for x in range(0, len(got), n):
                if not lib.item_masked(p0, p1, window, sinks, x, n):
                    assert all(set(got[x:x + n]) <= see[p] for p in see), (p0, x, n)


@pytest.mark.parametrize("seed", range(60))
def test_places_in_closed_form(lib, seed):
    rng = np.random.default_rng(seed)
    for _ in range(20):
        gq = int(rng.choice([1, 2, 3, 4, 7, 8, 16, 64, 100, 256]))
        rows = 256 if gq > 128 else int(rng.choice([128, 256]))
        n, ctx = int(rng.integers(1, 3000)), int(rng.choice([0, rng.integers(0, 200), rng.integers(0, 200000)]))
        window = int(rng.choice([0, 1, rng.integers(1, 300), rng.integers(1, 20000)]))
        sinks = int(rng.choice([0, 1, rng.integers(0, 300), rng.integers(0, 3000)]))
        assert lib.prefixes(n, ctx, gq, rows, window, sinks, int(rng.choice([0, 4]))) == 0


def test_places_of_the_longest_requests(lib):
    # 2^26 tokens, the longest a call takes: the sums stay within their types
    assert lib.prefixes(1 << 16, (1 << 26) - (1 << 16), 256, 256, 0, 0, 4) == 0
    assert lib.prefixes(1 << 16, (1 << 26) - (1 << 16), 256, 256, (1 << 26) - 1, 1 << 26, 4) == 0
    assert lib.prefixes(1 << 16, (1 << 26) - (1 << 16), 1, 128, 1, 0, 4) == 0


def split(lib, heads, gq, n, lens, window=0, sinks=0, max_q=None, max_len=None, nsm=152, rows=None):
    """(grid, chunks, slots read, holes, chunks computed twice or never, CTAs with work, most chunks of a CTA)."""
    max_q, max_len = max_q or max(max(n), 1), max_len or max(max(lens), 1)
    rows = rows or (8 if max_q * gq <= 8 else 128 if max_q * gq <= 128 else 256)
    out, ints = (ctypes.c_int * 6)(), ctypes.c_int * len(n)
    grid = lib.split(nsm, heads, gq, rows, max_q, max_len, window, sinks, len(n), ints(*n), ints(*lens), out)
    assert grid >= 1
    return (grid, *out)


@pytest.mark.parametrize("n,lens,opts", [
    ([1], [1], {}), ([1], [4096], {}), ([1], [4002], dict(window=1024, sinks=4)),
    ([4096], [4096], {}), ([2048], [32049], {}), ([2048], [32049], dict(window=1000, sinks=130)),
    ([1, 0, 509, 1, 0], [7000, 0, 509, 1, 900], dict(window=1024, sinks=16, max_q=4096, max_len=1 << 20)),
    ([0, 0, 1], [0, 5, 1], {}), ([1] * 200, [100 + 37 * i for i in range(200)], {}),
    ([1] * 300, [1] * 300, dict(max_len=1 << 20)), ([300], [300], dict(window=1)),
])
@pytest.mark.parametrize("heads,gq", [(1, 1), (8, 4), (4, 7), (2, 100), (1, 200)])
def test_batches(lib, heads, gq, n, lens, opts):
    grid, chunks, reads, holes, wrong, busy, most = split(lib, heads, gq, n, lens, **opts)
    assert holes == 0 and wrong == 0
    assert busy <= grid and chunks >= 1


@pytest.mark.parametrize("seed", range(300))
def test_drawn_batches(lib, seed):
    rng = np.random.default_rng(seed)
    reqs = int(rng.integers(1, 12))
    gq = int(rng.choice([1, 3, 4, 7, 8, 16, 150]))
    n = [int(rng.choice([0, 1, 1, rng.integers(1, 600)])) for _ in range(reqs)]
    if not any(n):
        n[0] = 1
    lens = [k + int(rng.choice([0, rng.integers(0, 300), rng.integers(0, 9000)])) for k in n]
    opts = dict(window=int(rng.choice([0, 1, rng.integers(1, 3000)])), sinks=int(rng.choice([0, 4, rng.integers(0, 400)])),
                nsm=int(rng.choice([1, 2, 7, 152])))
    if rng.random() < 0.4:
        opts.update(max_q=max(n) + int(rng.integers(0, 2000)), max_len=max(lens) + int(rng.integers(0, 100000)))
    grid, chunks, reads, holes, wrong, busy, most = split(lib, int(rng.choice([1, 2, 8])), gq, n, lens, **opts)
    assert holes == 0 and wrong == 0
