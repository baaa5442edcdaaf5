"""The tree attention's work split on the CPU, with the launch's own grid: whatever the call's bounds
(max_query_len, max_seq_len, the requests) are above the actual counts, the merge reads only slots that
this call wrote for that item, and every chunk is computed once.
"""
import ctypes
import os
import subprocess

import numpy as np
import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    so = str(tmp_path_factory.mktemp("split") / "tree_split.so")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", os.path.join(HERE, "tree_split_host.cpp"), "-o", so],
                   check=True, capture_output=True)
    return ctypes.CDLL(so)


def split(lib, heads, gq, n, lens, max_q=None, max_len=None, nsm=152, rows=None):
    """(grid, chunks, slots read, holes, chunks computed twice or never, CTAs with work, most chunks of a CTA)."""
    max_q, max_len = max_q or max(max(n), 1), max_len or max(max(lens), 1)
    rows = rows or (128 if max_q * gq <= 128 else 256)
    out, ints = (ctypes.c_int * 6)(), ctypes.c_int * len(n)
    grid = lib.split(nsm, heads, gq, rows, max_q, max_len, len(n), ints(*n), ints(*lens), out)
    assert grid >= 1
    return (grid, *out)


@pytest.mark.parametrize("n,lens,bounds", [
    ([8], [508], dict(max_len=4096)),                       # one user, a server's fixed bound: one place per CTA before
    ([8], [1500], dict(max_len=8192)), ([8], [700], dict(max_len=8192)),
    ([8, 8], [600, 400], dict(max_len=1000)),
    ([8, 5, 0, 8], [900, 20, 31, 130], {}),
    ([1], [129], dict(max_len=1 << 20)),                    # two chunks under the widest bound
    ([8], [700], dict(max_len=8192, max_q=256)),            # the kernel of two tiles with one tile's rows
    ([40, 8], [500, 300], dict(max_len=8192)),              # chunks of three and of four places
    ([256], [300], dict(max_len=8192)),
])
@pytest.mark.parametrize("heads", [1, 2, 8])
def test_small_batches_under_wide_bounds(lib, heads, n, lens, bounds):
    grid, chunks, reads, holes, wrong, busy, most = split(lib, heads, 4, n, lens, **bounds)
    assert holes == 0 and wrong == 0
    # spread over the CTAs there are: at most a chunk of three places more than an even share
    assert most <= -(-chunks // grid) + 1


@pytest.mark.parametrize("gq", [1, 4, 7])
@pytest.mark.parametrize("max_q", [8, 256])
def test_one_place_widths_are_not_doubled_up(lib, gq, max_q):
    # chunks of one width, fewer than CTAs: each in a CTA of its own
    for length in (128, 129, 700, 1500, 2400):
        grid, chunks, _, holes, wrong, busy, most = split(lib, 8, gq, [8], [length], max_q=max_q, max_len=8192)
        assert holes == 0 and wrong == 0 and chunks <= grid and busy == chunks and most == 1


@pytest.mark.parametrize("seed", range(600))
def test_the_merge_reads_what_this_call_wrote(lib, seed):
    rng = np.random.default_rng(seed)
    heads, gq = int(rng.choice([1, 2, 4, 8, 16])), int(rng.choice([1, 4, 7, 8]))
    reqs = int(rng.integers(1, int(rng.choice([3, 8, 40]))))
    n = rng.integers(0, int(rng.choice([2, 9, 65, 257])), reqs)
    n[int(rng.integers(0, reqs))] = max(int(n.max()), 1)
    lens = n + rng.integers(0, int(rng.choice([50, 900, 6000])), reqs)
    mq, ml = int(n.max()), int(lens.max())
    bounds = dict(max_q=int(rng.choice([mq, min(256, 2 * mq), 256])), max_len=int(rng.choice([ml, 4 * ml, max(ml, 8192)])),
                  nsm=int(rng.choice([1, 7, 50, 152])))
    grid, chunks, reads, holes, wrong, *_ = split(lib, heads, gq, n.tolist(), lens.tolist(), **bounds)
    assert wrong == 0
    assert holes == 0, (holes, reads)
