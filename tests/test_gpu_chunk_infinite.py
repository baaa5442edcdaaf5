"""Attention of chunks of new tokens where every score of a token is -inf: a softmax over nothing but -inf has no value, so
the token's output is NaN, as the oracle's is, in every kernel and in every way in which parts of an item are joined."""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_chunk import build, caches64, run
from test_gpu_kv_quant import built, handle, status  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu

CASES = [  # nq, nkv, t, ctx, n
    (8, 2, 2, [60], [1]), (8, 2, 2, [60, 5], [2, 1]),       # up to eight rows: whole items
    (8, 2, 2, [6001], [1]), (8, 2, 2, [6001], [2]),         # their parts joined by a kernel
    (8, 2, 2, [60], [30]), (8, 2, 2, [60], [90]),           # one tile and two, whole
    (8, 2, 2, [6001], [30]), (8, 2, 2, [6001], [90]),       # their parts joined by a kernel
    (8, 8, 1, [700] * 20, [30] * 20), (16, 8, 1, [700] * 20, [90] * 20),             # two or three parts of an item, joined by the CTAs
    (32, 8, 4, [9000] + [0] * 39, [30] + [1] * 39), (32, 8, 4, [9000] + [0] * 39, [70] + [1] * 39),   # more than eight parts
]


def below(x):
    """Element 0 of every head row made a negative number."""
    x = x.clone()
    if x.dtype is torch.float8_e4m3fn:
        x.view(torch.uint8)[..., 0] = 0xb8                   # -1
    else:
        x[..., 0] = -1
    return x


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (500, 3)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_a_token_whose_scores_are_all_minus_infinity(case, window, sinks, q8):
    nq, nkv, t, ctx, n = CASES[case]
    c = build(nq, nkv, t, ctx, n, 16, seed=200 + case, q8=q8)
    c["ck"] = below(c["ck"])
    h = handle(nq, nkv, t)
    want = run(h, c, window, sinks)[0].clone()
    assert torch.isfinite(want.float()).all()
    last = c["qsl"][1:] - 1                                   # every request's last token: q is +inf where k is negative
    q = c["qkv"].clone()
    q.view(t, c["T"], -1, 128)[:, last, :nq // t, 0] = float("inf")
    out, ws = run(h, dict(c, qkv=q), window, sinks)
    assert status(ws) == 0
    others = np.setdiff1d(np.arange(c["T"]), last)
    assert torch.equal(out[:, others], want[:, others])
    assert torch.isnan(out[:, last].float()).all()
    if sum(n) * sum(ctx) < 10 ** 6:
        ck, cv = caches64(c)
        ref = oracle.chunk_attention(oracle.bf16_to_f64(q), c["qsl"], c["lens"], c["tables"], ck, cv, nq, nkv, 128, t, c["bs"],
                                     window, sinks)
        assert np.isnan(ref[:, last]).all() and np.isfinite(ref[:, others]).all()


@pytest.mark.parametrize("case", [2, 3, 6, 7, 8, 9, 10, 11])
def test_keys_whose_scores_are_minus_infinity_have_no_weight(case):
    # the first half of every context, whole parts of items among it: as with a score that is as low as can be
    nq, nkv, t, ctx, n = CASES[case]
    c = build(nq, nkv, t, ctx, n, 16, seed=230 + case)
    q = c["qkv"].clone()
    q.view(t, c["T"], -1, 128)[:, :, :nq // t, 0] = 1.0
    outs = []
    for low in (-float("inf"), -2.0 ** 100):
        ck = c["ck"].clone()
        for b, x in enumerate(ctx):
            j = np.arange(x // 2)
            at = torch.from_numpy(c["tables"][b, j // 16] * 16 + j % 16)
            ck.view(t, -1, nkv // t, 128)[:, at, :, 0] = low
        out, ws = run(handle(nq, nkv, t), dict(c, qkv=q, ck=ck))
        assert status(ws) == 0 and torch.isfinite(out.float()).all()
        outs.append(out)
    assert torch.equal(*outs)
