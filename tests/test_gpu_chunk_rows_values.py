"""Attention of chunks of new tokens where a kv head has up to eight query rows: values that are not finite reach the tokens
that see them alone, and a wait that runs out."""
import numpy as np
import pytest
import torch

import oracle
import tensor_linear_layers_gb300 as tl
from test_gpu_chunk import build, check, run
from test_gpu_kv_quant import built, handle, status  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu

SIZES = [  # nq, nkv, t, ctx, n
    (8, 2, 2, [150, 5], [2, 2]), (4, 4, 2, [150, 5], [8, 3]), (7, 1, 1, [150, 5], [1, 1]),
    (8, 2, 2, [5000, 40], [2, 1]), (4, 4, 2, [5000, 40], [8, 3]),          # items in parts
]


def tainted(c, window, sinks, places):
    """Which tokens see one of the positions (request, position)."""
    seen = np.zeros(c["T"], dtype=bool)
    for b, j in places:
        for i in range(c["n"][b]):
            seen[c["qsl"][b] + i] |= bool(oracle.kv_quant.sees(c["lens"][b] - c["n"][b] + i, c["lens"][b], window, sinks)[j])
    return seen


def places_of(c, window):
    ends = [(b, x - 1) for b, x in enumerate(c["lens"])]     # every request's last token: seen by itself alone
    if window == 0:
        return ends
    # a key long past, one that leaves the window between two tokens, a sink
    first = c["lens"][0] - c["n"][0] - window + 1
    return ends + [(0, max(0, first)), (0, c["lens"][0] // 2), (1, 1)]


def past_the_ends(x, c, value):
    for b, L in enumerate(c["lens"]):
        if L % c["bs"]:
            x[:, c["tables"][b, L // c["bs"]], L % c["bs"]:] = value


@pytest.mark.parametrize("size", range(len(SIZES)))
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3), (2, 0), (1, 0)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_a_token_does_not_see_has_no_effect(size, window, sinks, bad):
    nq, nkv, t, ctx, n = SIZES[size]
    c = build(nq, nkv, t, ctx, n, 16, seed=400 + size)
    h = handle(nq, nkv, t)
    clean = run(h, c, window, sinks)[0].clone()
    check(clean, c, window, sinks)
    places = places_of(c, window)
    ck, cv = c["ck"].clone(), c["cv"].clone()
    for b, j in places:
        s = oracle.slot_of(c["tables"], b, j, 16)
        ck[:, s // 16, s % 16] = bad
        cv[:, s // 16, s % 16, :, 1::2] = bad
    past_the_ends(ck, c, bad)
    past_the_ends(cv, c, bad)
    hit = tainted(c, window, sinks, places)
    got, ws = run(h, dict(c, ck=ck, cv=cv), window, sinks)
    assert status(ws) == 0
    assert torch.equal(got[:, ~hit], clean[:, ~hit])
    # bad values in v alone reach the tokens that see them, in their own dimensions
    got, ws = run(h, dict(c, cv=cv), window, sinks)
    assert status(ws) == 0
    assert torch.equal(got[:, ~hit], clean[:, ~hit])
    g, w = (x.float().cpu().view(t, c["T"], -1, 64, 2) for x in (got, clean))
    assert not torch.isfinite(g[:, hit][..., 1]).any()
    assert torch.equal(g[:, hit][..., 0], w[:, hit][..., 0])


@pytest.mark.parametrize("size", range(len(SIZES)))
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3), (2, 0), (1, 0)])
@pytest.mark.parametrize("which", ["sk", "sv"])
def test_rows_of_the_8_bit_cache_that_stand_for_nan(size, window, sinks, which):
    nq, nkv, t, ctx, n = SIZES[size]
    c = build(nq, nkv, t, ctx, n, 16, seed=420 + size, q8=True)
    h = handle(nq, nkv, t)
    clean = run(h, c, window, sinks)[0].clone()
    check(clean, c, window, sinks)
    places = places_of(c, window)
    scales = c[which].clone()
    for b, j in places:
        s = oracle.slot_of(c["tables"], b, j, 16)
        scales[:, s // 16, s % 16] = 255
    past_the_ends(scales, c, 255)
    hit = tainted(c, window, sinks, places)
    got, ws = run(h, dict(c, **{which: scales}), window, sinks)
    assert status(ws) == 0
    assert torch.equal(got[:, ~hit], clean[:, ~hit])
    assert torch.isnan(got[:, hit].float()).all()


@pytest.mark.parametrize("q8", [False, True])
def test_wait_limit_runs_out_and_context_survives(q8):
    # a call of many requests without new tokens: the warps that wait for the first segment wait as long as one
    # goes through all of them (some ms), the only wait of this kernel that lasts
    reqs = 60000
    c = build(8, 2, 2, [700], [1], 16, seed=430, q8=q8)
    h = handle(8, 2, 2)
    many = dict(c, tables=np.repeat(c["tables"], reqs, 0), lens=[0] * (reqs - 1) + [701], n=[0] * (reqs - 1) + [1],
                qsl=np.array([0] * reqs + [1]))
    good, ws = run(h, many)
    good = good.clone()
    assert status(ws) == 0
    check(good, c)
    tl.set_wait_timeout(1)                                  # waits of more than one suspended try (20 us) run out
    try:
        _, ws = run(h, many, ws=ws)
        st = status(ws)                                     # returns: nothing hung, nothing faulted
    finally:
        tl.set_wait_timeout(2_000_000_000)
    assert st == tl.TP_ERR_TIMEOUT
    ws.zero_()
    out, ws = run(h, many, ws=ws)
    assert status(ws) == 0 and torch.equal(out, good)
