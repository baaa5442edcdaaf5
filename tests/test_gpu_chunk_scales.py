"""Attention of chunks of new tokens over an 8-bit cache where scales and queries are far from one: every kernel gives the
oracle's result."""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_chunk import build, caches64, run
from test_gpu_kv_quant import built, handle, status  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu


def check(got, c, window=0, sinks=0):
    """Within what the roundings allow: those of test_gpu_chunk.check, and, in the kernel for up to eight rows, those of the
    f16 weights w_j = 2^(x_j - m), x_j the score's exponent and v's scale together, the largest at 2^7 or more where
    some v has a scale of 2^-86 or more, at 2^-7 or more where none has. Under f16's normal numbers a weight is off by
    2^-25 at most: 2^-32 of the largest (2^-18), times 448 in O for each of the keys."""
    nq, nkv, t = c["heads"]
    ck, cv = caches64(c)
    ref, size, spread, score = oracle.chunk_attention(oracle.bf16_to_f64(c["qkv"]), c["qsl"], c["lens"], c["tables"], ck, cv,
                                                      nq, nkv, 128, t, c["bs"], window, sinks, bound=True)
    top = int(c["sv"].max()) - 127
    lost = max(c["lens"]) * (2.0 ** -109 * np.abs(cv).max() + 2.0 ** (-32 + max(0, -86 - top)) * 448 * 2.0 ** top)
    off = 4 * 130 * 2.0 ** -24 * np.repeat(score, 128, -1) + 2.0 ** -20 + (max(c["lens"]) / 16 + 8) * 2.0 ** -22
    tol = 2.0 ** -8 * (np.minimum(size, 7 * spread) * (1 + 2.0 ** -8) + np.abs(ref)) + off * size + lost
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all()
    err = np.abs(g - ref) - tol
    assert err.max() <= 0, f"over by {err.max():.3e} at {np.unravel_index(err.argmax(), err.shape)}, tolerance {tol.min():.3e}"
    return ref


SIZES = [([200], [1]), ([200], [2]), ([5000], [2]), ([200], [20]), ([5000], [150])]    # up to eight rows, one tile, two


@pytest.mark.parametrize("ctx,n", SIZES)
@pytest.mark.parametrize("end,sk", [(27, 127), (245, 127), (140, 135), (127, 140), (41, 127), (0, 127)])
def test_both_ends_of_the_scales(ctx, n, end, sk):
    # v rows of 2^-100 and 2^118 times a code, also none but rows that were never written (byte 0, codes 0); and k rows
    # whose second factor is not one
    c = build(4, 2, 1, ctx, n, 16, seed=end, q8=True)
    c["sv"] = torch.full_like(c["sv"], end)
    if end == 0:
        c["cv"] = torch.zeros_like(c["cv"].view(torch.uint8)).view(torch.float8_e4m3fn)
    c["sk"] = torch.full_like(c["sk"], sk if sk > 134 else sk - 8)        # codes reach 448: keep the scores moderate
    if sk > 134:
        c["qkv"] = (c["qkv"].float() * 2.0 ** (119 - sk)).to(torch.bfloat16)
    out, ws = run(handle(4, 2, 1), c)
    assert status(ws) == 0
    check(out, c)


@pytest.mark.parametrize("ctx,n", SIZES)
@pytest.mark.parametrize("power", [-100, -60, 60, 100, 114])
def test_scales_of_k_that_a_query_makes_up_for(ctx, n, power):
    # q of 2^-power against k of 2^power: moderate scores
    c = build(4, 2, 1, ctx, n, 16, seed=300 + power, q8=True)
    c["sk"] = torch.full_like(c["sk"], 119 + power)
    c["qkv"] = (c["qkv"].float() * 2.0 ** -power).to(torch.bfloat16)
    out, ws = run(handle(4, 2, 1), c)
    assert status(ws) == 0
    check(out, c)


@pytest.mark.parametrize("ctx,n", SIZES)
@pytest.mark.parametrize("q,k", [(60, 90), (39, 118), (118, 118)])
def test_products_of_zero_of_large_queries_and_large_scales(ctx, n, q, k):
    # k has codes of 0 wherever q is not 0: every score is 0, however large both factors are
    c = build(4, 2, 1, ctx, n, 16, seed=310, q8=True)
    c["sk"] = torch.full_like(c["sk"], 127 + k)
    c["ck"] = c["ck"].clone()
    c["ck"].view(torch.uint8)[..., 64:] = 0
    c["qkv"] = (c["qkv"].float().clamp(-3, 3) * 2.0 ** q).to(torch.bfloat16)
    c["qkv"].view(1, c["T"], -1, 128)[..., :64] = 0
    out, ws = run(handle(4, 2, 1), c)
    assert status(ws) == 0
    check(out, c)


@pytest.mark.parametrize("ctx,n", SIZES + [([40, 700], [1, 2]), ([20000], [1])])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 20)])
def test_slots_that_were_never_written_count_as_zeros(ctx, n, window, sinks):
    # a cache as kv_quant_cache makes it, some of its pages without a write (byte 0 and codes 0): keys and values of 0,
    # which have weight like any others, whole warps' keys and whole parts of items among them
    bs = 16
    c = build(4, 2, 1, ctx, n, bs, seed=330 + len(ctx), q8=True)
    rng = np.random.default_rng(5)
    for name in ("ck", "cv", "sk", "sv"):
        c[name] = c[name].clone()
    for b, x in enumerate(ctx):
        pages = np.nonzero(rng.random(x // bs) < 0.4)[0]
        pages = np.unique(np.concatenate([[1], pages, np.arange(x // bs // 2, x // bs // 2 + x // bs // 5)]))
        at = torch.from_numpy(c["tables"][b, pages])
        for name in ("ck", "cv", "sk", "sv"):
            c[name].view(torch.uint8)[:, at] = 0
    out, ws = run(handle(4, 2, 1), c, window, sinks)
    assert status(ws) == 0
    check(out, c, window, sinks)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("ctx,n", SIZES[:4] + [([900], [70])])
def test_scores_of_millions(ctx, n, q8):
    # scores up to 2^22, the largest that the interface names: the key with the largest takes all the weight. A score is off by
    # 130 * 2^-24 of its products' sizes at most, far less than the two largest differ by (asserted); the weight's
    # rounding to bf16 and the output's are 2^-8 each.
    c = build(4, 2, 1, ctx, n, 16, seed=390 + n[0], q8=q8)
    ck = caches64(c)[0]
    heads = oracle.bf16_to_f64(c["qkv"]).reshape(c["T"], -1, 128)[:, :4]
    slots = [oracle.slot_of(c["tables"], 0, j, 16) for j in range(c["lens"][0])]
    keys = ck[0].reshape(-1, 2, 128)[slots].repeat(2, 1)
    score = np.einsum("ihd,jhd->ihj", heads, keys) / np.sqrt(128)
    power = int(np.floor(np.log2(2.0 ** 22 / np.abs(score).max())))
    c["qkv"] = (c["qkv"].float() * 2.0 ** power).to(torch.bfloat16)
    score *= 2.0 ** power
    score[~(np.arange(c["lens"][0]) <= ctx[0] + np.arange(n[0])[:, None])[:, None].repeat(4, 1)] = -np.inf
    best = np.sort(score, -1)[..., -2:]
    size = np.einsum("ihd,jhd->ihj", np.abs(heads), np.abs(keys)).max() * 2.0 ** power / np.sqrt(128)
    assert (best[..., 1] - best[..., 0]).min() > 4 * 130 * 2.0 ** -24 * size + 30
    out, ws = run(handle(4, 2, 1), c)
    assert status(ws) == 0
    ref = oracle.chunk_attention(oracle.bf16_to_f64(c["qkv"]), c["qsl"], c["lens"], c["tables"], *caches64(c), 4, 2, 128, 1, 16)
    assert (np.abs(out.double().cpu().numpy() - ref) <= (2 * 2.0 ** -8 + 2.0 ** -15) * np.abs(ref)).all()


@pytest.mark.parametrize("exponent", [20, -20, 1])
def test_a_scale_of_v_beside_a_large_score(exponent):
    # requests of one token, which attends to itself: its output is its v, whatever the score is. Scores times log2(e) lie
    # on both sides of 2^22, in steps of 1/4, where a sum with v's exponent loses a bit of them or more. The weight is
    # rounded to f16 (2^-11 of it) and comes from an exponential that is good to 2^-20, the output is rounded to bf16.
    reqs = 128
    c = build(4, 2, 1, [0] * reqs, [1] * reqs, 16, seed=335, q8=True)
    c["sv"] = torch.full_like(c["sv"], 127 + exponent)
    c["sk"] = torch.full_like(c["sk"], 127)
    c["ck"] = torch.full_like(c["ck"].view(torch.uint8), 0x38).view(torch.float8_e4m3fn)     # k = 1
    q = torch.zeros(1, reqs, 4, 128)
    for b in range(reqs):
        rest = (2.0 ** 22 - 16 + b / 4) * np.sqrt(128) / np.log2(np.e)
        for i in range(4):                                    # the score as a sum of four bf16 numbers
            x = float(torch.tensor(rest).to(torch.bfloat16))
            q[0, b, :, i] = x
            rest -= x
    c["qkv"].view(1, reqs, 8, 128)[:, :, :4] = q.to(torch.bfloat16)
    out, ws = run(handle(4, 2, 1), c)
    assert status(ws) == 0
    v = caches64(c)[1]
    slots = [oracle.slot_of(c["tables"], b, 0, 16) for b in range(reqs)]
    want = v.reshape(-1, 2, 128)[slots].repeat(2, 1).reshape(1, reqs, 512)
    assert (np.abs(out.double().cpu().numpy() - want) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(want)).all()
