"""Attention of chunks of new tokens where an item of one or two tiles of query rows is computed in parts by several CTAs:
values that are not finite reach the tokens that see them alone, however the parts are joined."""
import pytest
import torch

import oracle
from test_gpu_chunk import build, run
from test_gpu_chunk_rows_values import past_the_ends, places_of, tainted
from test_gpu_kv_quant import built, handle, status  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu

SIZES = [  # nq, nkv, t, ctx, n
    (8, 2, 2, [5000, 40], [30, 9]), (8, 2, 2, [5000, 40], [90, 40]),       # joined by a kernel
    (8, 8, 1, [700] * 20, [30] * 20), (16, 8, 1, [700] * 20, [90] * 20), # two or three parts, joined by the CTAs
    (32, 8, 4, [9000] + [3] * 39, [30] + [1] * 39),                       # more than eight of them
]


@pytest.mark.parametrize("size", range(len(SIZES)))
@pytest.mark.parametrize("window,sinks", [(0, 0), (600, 3)])
@pytest.mark.parametrize("bad", [float("nan"), -float("inf"), "scales"])
def test_what_a_token_does_not_see_has_no_effect(size, window, sinks, bad):
    nq, nkv, t, ctx, n = SIZES[size]
    q8 = bad == "scales"
    c = build(nq, nkv, t, ctx, n, 16, seed=440 + size, q8=q8)
    h = handle(nq, nkv, t)
    clean = run(h, c, window, sinks)[0].clone()
    places = places_of(c, window)
    hit = tainted(c, window, sinks, places)
    for names in (["k", "v"], ["v"]):
        d = dict(c)
        for x in names:
            name, value = ("s" + x, 255) if q8 else ("c" + x, bad)
            d[name] = c[name].clone()
            for b, j in places:
                s = oracle.slot_of(c["tables"], b, j, 16)
                d[name][:, s // 16, s % 16] = value
            past_the_ends(d[name], c, value)
        got, ws = run(h, d, window, sinks)
        assert status(ws) == 0
        assert torch.equal(got[:, ~hit], clean[:, ~hit])
    assert not torch.isfinite(got[:, hit].float()).any()     # (v alone)
