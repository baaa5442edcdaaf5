"""Accepted paths of more than 256 tokens (the kernel goes through a list in strips of 256) and lists that end badly
at a strip's edge (tp_kv_cache_compact): copies, bit for bit.
"""
import numpy as np
import pytest

import oracle
import tensor_linear_layers_gb300 as tl
from test_gpu_kv_pages import bits, built, compact_case, handle, run_compact, status  # noqa: F401 (built: a fixture)

pytestmark = pytest.mark.gpu


def equal(h, c, ctx, kept, bs, want):
    before = [bits(x) for x in c["ck"] + c["cv"]]
    new, ws = run_compact(h, c)
    assert status(ws) == want
    assert new.tolist() == [x + len(a) for x, a in zip(ctx, kept)]
    for a, b in zip(before, c["ck"] + c["cv"]):
        np.testing.assert_array_equal(bits(b), oracle.compact(a, ctx, kept, c["src"], c["dst"], bs))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("m", [None, 1000])
def test_lists_of_several_strips(in_place, m):
    rng = np.random.default_rng(5)
    n, keep = [600, 256, 700, 900, 257], [300, 256, 513, 600, 257]
    ctx = [0, 13, 40, 7, 255]
    accepted = [sorted(rng.permutation(k)[:a].tolist()) for k, a in zip(n, keep)]
    accepted[2] = list(range(1, 514))                       # a shift by one over all strips
    h, bs = handle(8, 2, 2), 16
    equal(h, compact_case(h, ctx, n, accepted, bs, 2, 31, in_place, m), ctx, accepted, bs, 0)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("at", [255, 256, 257, 511, 512])
def test_lists_that_end_badly_at_an_edge(in_place, at):
    n, ctx, bs = [600, 600, 600], [3, 20, 9], 16
    h = handle(8, 2, 2)
    lists = [list(range(2, 582))] * 3
    c = compact_case(h, ctx, n, lists, bs, 1, at, in_place)
    c["acc"][0, at] = c["acc"][0, at - 1]                   # does not rise
    c["acc"][1, at] = 600                                   # past the drafts
    c["acc"][2, at] = -1                                    # the end; what follows is not looked at
    c["acc"][2, at + 1] = 10_000
    kept = [x[:at] for x in lists]
    equal(h, c, ctx, kept, bs, tl.TP_ERR_SHAPE)


def test_a_strip_that_ends_the_list_is_no_error():
    n, ctx, bs = [600, 600], [3, 20], 16
    h = handle(8, 2, 2)
    lists = [list(range(2, 258)), list(range(1, 513))]      # 256 and 512 tokens, then the end
    equal(h, compact_case(h, ctx, n, lists, bs, 1, 77, True, m=580), ctx, lists, bs, 0)
