"""Attention of chunks of new tokens over the paged cache (tp_chunk_attention) against the float64 oracle: bf16 and
8-bit caches, windows and sinks, decoding requests and prompts in one call."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import tensor_linear_layers_gb300 as tl
from test_gpu_kv_quant import built, dev, handle, status  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu


def build(nq, nkv, t, ctx, n, bs, seed, q8=False, pad=0, extra=3, scale=1.0):
    """A call's arrays on the CPU; tables hold an id out of range wherever no page is needed."""
    g, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    q_per, kv_per, _ = oracle.gqa_partition(nq, nkv, t)
    lens = [c + k for c, k in zip(ctx, n)]
    need = [-(-x // bs) for x in lens]
    blocks = sum(need) + extra
    perm = rng.permutation(blocks)
    tables = np.full((len(n), max(max(need), 1) + 1), -1, dtype=np.int64)
    at = 0
    for b, k in enumerate(need):
        tables[b, :k] = perm[at:at + k]
        at += k
    qsl = np.concatenate([[0], np.cumsum(n)])
    T = int(qsl[-1]) + pad
    qkv = (torch.randn(t, T, (q_per + 2 * kv_per) * 128, generator=g) * scale).to(torch.bfloat16)
    caches = [torch.randn(t, blocks, bs, kv_per, 128, generator=g).to(torch.bfloat16) for _ in range(2)]
    c = dict(qkv=qkv, qsl=qsl, lens=lens, tables=tables, n=list(n), T=T, bs=bs, heads=(nq, nkv, t), sk=None, sv=None)
    if q8:
        mags = oracle.e4m3_values()[:127]
        for name, x in zip("kv", caches):
            x = x.float() * torch.exp(2 * torch.randn(x.shape[:-1], generator=g))[..., None] * (0.3 if name == "k" else 1)
            y, s = oracle.quantise(x.to(torch.bfloat16).double().numpy())
            code = (np.searchsorted(mags, np.abs(y)) + 128 * (y < 0)).astype(np.uint8)
            c["c" + name], c["s" + name] = torch.from_numpy(code).view(torch.float8_e4m3fn), torch.from_numpy(s.astype(np.uint8))
    else:
        c["ck"], c["cv"] = caches
    return c


def run(h, c, window=0, sinks=0, out=None, max_q=None, max_len=None, ws=None, **kw):
    cuda = {k: None if c[k] is None else c[k].cuda() for k in ("qkv", "ck", "cv", "sk", "sv")}
    return h.chunk_attention(cuda["qkv"], dev(c["qsl"]), dev(c["lens"]), dev(c["tables"]), cuda["ck"], cuda["cv"],
                             max_q or max(max(c["n"]), 1), max_len or max(max(c["lens"]), 1), window, sinks, cuda["sk"],
                             cuda["sv"], out=out, ws=ws, **kw)


def caches64(c):
    if c["sk"] is None:
        return oracle.bf16_to_f64(c["ck"]), oracle.bf16_to_f64(c["cv"])
    v = oracle.e4m3_values()
    return [oracle.values(v[c["c" + x].view(torch.uint8).numpy()], c["s" + x].numpy()) for x in "kv"]


def check(got, c, window=0, sinks=0):
    """Within what the roundings allow. P is rounded to bf16, 2^-8 of each weight at most: together at most 2^-8 sum p |v|,
    and, as they are independent, over 7 * 2^-8 sqrt(sum p^2 v^2) with a probability of 2 exp(-7^2 / 2) < 5e-11 only
    (Hoeffding). The output is rounded to bf16, 2^-8 of it. A score is a sum of 128 products in fp32, off by at most
    130 * 2^-24 of their sizes' sum (chopped additions: twice that), which changes a weight by twice as much at most,
    relative; the exponential and the weights' sum add 2^-20. O is a sum in fp32 of 16 products a step (chopped,
    2^-22 of the sizes' sum a step at most). Weights under fp32's smallest normal number, 2^-126, are taken as 0: the
    largest is held at 2^-17 or more (m is at most 17 above the largest exponent), so each is under 2^-109 of the sum of
    the weights, and all that is lost is under 2^-109 sum |v| (elements whose value is far below that are 0: where the one
    key that a token attends to has a v of exactly 0, the true value is what the others leave, down to 1e-86)."""
    nq, nkv, t = c["heads"]
    ck, cv = caches64(c)
    ref, size, spread, score = oracle.chunk_attention(oracle.bf16_to_f64(c["qkv"]), c["qsl"], c["lens"], c["tables"], ck, cv,
                                                      nq, nkv, 128, t, c["bs"], window, sinks, bound=True)
    off = 4 * 130 * 2.0 ** -24 * np.repeat(score, 128, -1) + 2.0 ** -20 + (max(c["lens"]) / 16 + 8) * 2.0 ** -22
    lost = 2.0 ** -109 * max(c["lens"]) * np.nanmax(np.where(np.isinf(cv), np.nan, np.abs(cv)))
    tol = 2.0 ** -8 * (np.minimum(size, 7 * spread) * (1 + 2.0 ** -8) + np.abs(ref)) + off * size + lost
    g = got.double().cpu().numpy()
    own = slice(0, int(c["qsl"][-1]))
    assert np.isfinite(g[:, own]).all()
    err = np.abs(g - ref)[:, own] - tol[:, own]
    assert err.max() <= 0, f"over by {err.max():.3e} at {np.unravel_index(err.argmax(), err.shape)}"
    return ref, tol


CASES = [  # nq, nkv, t, ctx, n, block size
    (8, 2, 2, [0], [1], 16),
    (8, 2, 2, [127], [1], 16), (8, 2, 2, [128], [1], 16),
    (4, 4, 1, [300, 0, 5, 40], [1, 1, 0, 1], 1),
    (32, 8, 4, [255, 1000, 17], [1, 1, 1], 16),
    (64, 1, 1, [700], [2], 24),                             # 64 q heads of a kv head: 128 rows
    (64, 1, 1, [200], [5], 24),                             # two tokens of 128 rows per group
    (7, 1, 1, [100], [300], 32),                            # 36 tokens of 7 heads per group, a last one of 12
    (9, 3, 1, [64, 3], [130, 50], 130),                     # three heads: 85 tokens per group, pages wider than a chunk
    (8, 2, 2, [0], [513], 16), (8, 2, 8, [200], [257], 16), # 8 shards of 2 kv heads
    (4, 4, 2, [0, 513, 90, 0, 1], [257, 1, 64, 0, 300], 8),
    (200, 1, 1, [90], [3], 16),                             # one token of 200 rows per group
]


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (100, 3), (129, 130)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_matches_oracle(case, window, sinks, q8):
    nq, nkv, t, ctx, n, bs = CASES[case]
    c = build(nq, nkv, t, ctx, n, bs, seed=case, q8=q8)
    out, ws = run(handle(nq, nkv, t), c, window, sinks)
    assert status(ws) == 0
    check(out, c, window, sinks)


@pytest.mark.parametrize("q8", [False, True])
def test_gathered_layout(q8):
    c = build(8, 2, 2, [40, 0], [30, 200], 16, seed=90, q8=q8)
    want, _ = run(handle(8, 2, 2), c, 64, 2)
    cg = dict(c, qkv=c["qkv"].permute(1, 0, 2).reshape(c["T"], -1).contiguous())
    out, ws = run(handle(8, 2, 2, tl.TP_FLAG_GATHERED), cg, 64, 2)
    assert status(ws) == 0
    assert torch.equal(out.view(c["T"], 2, -1).permute(1, 0, 2), want)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1000, 4), (2500, 300)])
def test_long_contexts_split_over_the_gpu(window, sinks, q8):
    # items that several CTAs compute in parts: one token, a few, and more than one group
    for n in ([1], [1, 3], [90, 1]):
        c = build(8, 2, 2, [6001, 3000][:len(n)], n, 16, seed=91 + len(n), q8=q8)
        out, ws = run(handle(8, 2, 2), c, window, sinks)
        assert status(ws) == 0
        check(out, c, window, sinks)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("n", [3, 30, 70, 200])
def test_one_long_request_among_many_short_ones(n, q8):
    # the call has an item and more for every SM, but the long request's items lie on a dozen SMs each, whose parts the
    # last of them joins
    c = build(32, 8, 2, [20000] + [0] * 39, [n] + [1] * 39, 16, seed=94, q8=q8)
    h = handle(32, 8, 2)
    out, ws = run(h, c)
    assert status(ws) == 0
    check(out, c)
    for _ in range(10):
        again, ws = run(h, c, ws=ws)
        assert status(ws) == 0 and torch.equal(again, out)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("nq,n,ctx,reqs,window,sinks", [
    (8, 100, 1092, 64, 0, 0),              # one head per row tile, the new tokens at the end of a chunk
    (8, 100, 1100, 64, 0, 0), (8, 128, 1024, 64, 0, 0), (8, 2, 1024, 90, 0, 0), (8, 120, 1030, 64, 700, 3),
    (32, 50, 1000, 40, 0, 0), (32, 60, 1024, 40, 600, 130), (32, 1, 900, 90, 0, 0),
])
def test_items_in_a_row(nq, n, ctx, reqs, window, sinks, q8):
    # several whole items one after another on every SM: the next one's keys come while the last one's values,
    # looked over, are handed on. The requests read the same pages: each has the one request's result.
    c = build(nq, 8, 1, [ctx], [n], 16, seed=100, q8=q8)
    many = dict(c, tables=np.repeat(c["tables"], reqs, 0), lens=[ctx + n] * reqs, qsl=np.arange(reqs + 1) * n, n=[n] * reqs,
                T=reqs * n, qkv=c["qkv"].repeat(1, reqs, 1))
    h = handle(nq, 8, 1)
    out, ws = run(h, many, window, sinks)
    assert status(ws) == 0
    one = out.view(1, reqs, n, -1)
    ref, tol = check(one[:, 0], c, window, sinks)
    err = (one.double().cpu() - torch.from_numpy(ref)[:, None]).abs() - torch.from_numpy(tol)[:, None]
    assert float(err.max()) <= 0
    for _ in range(3):
        assert torch.equal(out, run(h, many, window, sinks, ws=ws)[0])


@pytest.mark.parametrize("q8", [False, True])
def test_many_requests_and_runs_of_empty_ones(q8):
    nq, nkv, t = 4, 2, 1
    rng = np.random.default_rng(9)
    n, ctx = [0] * 300, [0] * 300
    for b in (0, 31, 32, 127, 128, 200, 299):
        n[b], ctx[b] = int(rng.integers(1, 90)), int(rng.integers(0, 400))
    for b in range(250, 298):
        ctx[b] = 17                                         # cached tokens, nothing new
    c = build(nq, nkv, t, ctx, n, 16, seed=50, q8=q8)
    out, ws = run(handle(nq, nkv, t), c, 70, 5)
    assert status(ws) == 0
    check(out, c, 70, 5)
    # nobody has a new token: nothing is computed, nothing written
    d = dict(c, qsl=np.zeros(301, dtype=np.int64), lens=ctx)
    keep = torch.full_like(out, 5.0)
    _, ws = run(handle(nq, nkv, t), d, out=keep, max_q=5, max_len=max(c["lens"]))
    assert status(ws) == 0 and (keep == 5.0).all()


def test_rows_of_no_request_are_left_as_they_were():
    c = build(8, 2, 2, [100, 30], [6, 3], 16, seed=8, pad=5)
    out = torch.full((2, 14, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    _, ws = run(handle(8, 2, 2), c, out=out)
    assert status(ws) == 0 and (out[:, 9:] == 5.0).all()
    check(out, c)


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3), (1, 0)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("wide", [False, True])
def test_what_a_token_does_not_see_has_no_effect(window, sinks, bad, wide):
    # k and v that are not finite: at a cached key, at new tokens, and past the requests' ends
    nq, nkv, t, bs = 8, 2, 2, 16
    n = [90, 40] if wide else [30, 9]
    c = build(nq, nkv, t, [150, 5], n, bs, seed=12)
    h = handle(nq, nkv, t)
    clean = run(h, c, window, sinks)[0].clone()
    ck, cv = c["ck"].clone(), c["cv"].clone()
    tainted = np.zeros(c["T"], dtype=bool)
    for b, j in ((0, 2), (0, 100), (0, 155), (1, 5 + n[1] // 2)):
        s = oracle.slot_of(c["tables"], b, j, bs)
        ck[:, s // bs, s % bs] = bad
        cv[:, s // bs, s % bs, :, 1::2] = bad
        for i in range(n[b]):
            p = c["lens"][b] - n[b] + i
            if j <= p and (window == 0 or j > p - window or j < sinks):
                tainted[c["qsl"][b] + i] = True
    for b, L in enumerate(c["lens"]):                       # the last page past the request's tokens
        if L % bs:
            ck[:, c["tables"][b, L // bs], L % bs:] = bad
            cv[:, c["tables"][b, L // bs], L % bs:] = bad
    got, ws = run(h, dict(c, ck=ck, cv=cv), window, sinks)
    assert status(ws) == 0
    assert torch.equal(got[:, ~tainted], clean[:, ~tainted]) and (window == 0 or not tainted.all())
    # bad values in v alone reach the tokens that see them, in their own dimensions
    got, ws = run(h, dict(c, cv=cv), window, sinks)
    g = got.float().cpu().view(2, c["T"], 4, 64, 2)
    assert status(ws) == 0
    assert torch.equal(got[:, ~tainted], clean[:, ~tainted])
    assert not torch.isfinite(g[:, tainted][..., 1]).any()
    assert torch.equal(g[:, tainted][..., 0], clean.float().cpu().view(2, c["T"], 4, 64, 2)[:, tainted][..., 0])


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3), (1, 0)])
@pytest.mark.parametrize("wide", [False, True])
def test_rows_of_the_8_bit_cache_that_stand_for_nan(window, sinks, wide):
    nq, nkv, t, bs = 8, 2, 2, 16
    n = [90, 40] if wide else [30, 9]
    c = build(nq, nkv, t, [150, 5], n, bs, seed=13, q8=True)
    h = handle(nq, nkv, t)
    clean = run(h, c, window, sinks)[0].clone()
    for which in ("sk", "sv"):
        sc = c[which].clone()
        tainted = np.zeros(c["T"], dtype=bool)
        for b, j in ((0, 2), (0, 100), (0, 155), (1, 5 + n[1] // 2)):
            s = oracle.slot_of(c["tables"], b, j, bs)
            sc[:, s // bs, s % bs] = 255
            for i in range(n[b]):
                p = c["lens"][b] - n[b] + i
                if j <= p and (window == 0 or j > p - window or j < sinks):
                    tainted[c["qsl"][b] + i] = True
        for b, L in enumerate(c["lens"]):
            if L % bs:
                sc[:, c["tables"][b, L // bs], L % bs:] = 255
        got, ws = run(h, dict(c, **{which: sc}), window, sinks)
        assert status(ws) == 0
        assert torch.equal(got[:, ~tainted], clean[:, ~tainted])
        assert torch.isnan(got[:, tainted].float()).all()


def test_scales_at_both_ends_of_their_range():
    # v rows of 2^-100 and 2^118 times a code, and k rows whose second factor is not one (scale bytes over 134)
    nq, nkv, t = 4, 2, 1
    for end, sk in ((27, 127), (245, 127), (140, 135), (127, 140)):
        c = build(nq, nkv, t, [200], [20], 16, seed=end, q8=True)
        c["sv"] = torch.full_like(c["sv"], end)
        c["sk"] = torch.full_like(c["sk"], sk - 8)            # codes reach 448: keep the scores moderate
        if sk > 134:
            c["sk"] = torch.full_like(c["sk"], sk)
            c["qkv"] = (c["qkv"].float() * 2.0 ** (119 - sk)).to(torch.bfloat16)
        out, ws = run(handle(nq, nkv, t), c)
        assert status(ws) == 0
        check(out, c)


def test_large_scores_and_equal_bits_on_repetition():
    for q8 in (False, True):
        c = build(16, 4, 2, [1500, 70, 900], [12, 130, 1], 16, seed=21, q8=q8, scale=4.0)
        h = handle(16, 4, 2)
        ws = torch.zeros(h.chunk_attention_workspace_size(3, 130, 1512), dtype=torch.uint8, device="cuda")
        a = run(h, c, 600, 2, ws=ws)[0].clone()
        check(a, c, 600, 2)
        for _ in range(3):
            assert torch.equal(a, run(h, c, 600, 2, ws=ws)[0])
        assert status(ws) == 0


def test_one_workspace_for_calls_of_other_bounds():
    # what an earlier call left in the slots is never read
    h = handle(8, 2, 2)
    ws = torch.zeros(h.chunk_attention_workspace_size(4, 300, 9000), dtype=torch.uint8, device="cuda")
    calls = [([3000, 10, 0, 700], [1, 300, 1, 7], False, 0, 0), ([8000], [1], True, 0, 0), ([8000], [1], True, 500, 4),
             ([500, 600], [2, 1], False, 0, 0), ([0], [300], True, 90, 0)]
    for k, (ctx, n, q8, window, sinks) in enumerate(calls + calls[::-1]):
        c = build(8, 2, 2, ctx, n, 16, seed=60 + k, q8=q8)
        for bounds in ({}, dict(max_q=300, max_len=9000)):
            if bounds:
                c["tables"] = np.pad(c["tables"], ((0, 0), (0, 563 - c["tables"].shape[1])), constant_values=-1)
            out, _ = run(h, c, window, sinks, ws=ws, **bounds)
            assert status(ws) == 0
            check(out, c, window, sinks)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("nq,nkv,t", [(8, 2, 2), (7, 1, 1), (64, 1, 1), (32, 8, 4)])
def test_a_workspace_of_larger_bounds_serves_smaller_ones(nq, nkv, t, q8):
    h = handle(nq, nkv, t)
    bounds = [(r, q, m) for r in (1, 3, 100) for q in (1, 2, 3, 20, 40, 300) for m in (300, 5000)]
    size = {b: h.chunk_attention_workspace_size(*b) for b in bounds}
    for a in bounds:
        for b in bounds:
            if all(x <= y for x, y in zip(a, b)):
                assert size[a] <= size[b], (a, b)
    # and the calls of them all in one, in turn, with the results of workspaces of their own
    ws = torch.zeros(size[(100, 300, 5000)], dtype=torch.uint8, device="cuda")
    calls = [build(nq, nkv, t, ctx, n, 16, seed=i, q8=q8) for i, (ctx, n) in enumerate((
        ([2000], [1]), ([2000, 70], [2, 1]), ([3000], [300]), ([40] * 100, [1] * 100), ([400] * 20, [3] * 20), ([4000], [20])))]
    want = [run(h, c, 900, 5)[0] for c in calls]
    for _ in range(2):
        for c, x in zip(calls, want):
            out, _ = run(h, c, 900, 5, ws=ws)
            assert status(ws) == 0 and torch.equal(out, x)


def test_workspace_and_output_on_16_byte_boundaries():
    for nq, nkv, t, n in ((8, 2, 4, 9), (4, 4, 2, 5), (9, 3, 1, 43), (9, 3, 1, 9)):
        c = build(nq, nkv, t, [700, 64], [n, 2], 16, seed=n)
        h = handle(nq, nkv, t)
        need = h.chunk_attention_workspace_size(2, n, 700 + n)
        buf = torch.zeros(need + 64, dtype=torch.uint8, device="cuda")
        buf[16 + need:] = 77
        out = torch.empty(c["T"] * nq * 128 + 8, dtype=torch.bfloat16, device="cuda")[8:].view(t, c["T"], -1)
        _, ws = run(h, c, ws=buf[16:16 + need], out=out)
        assert status(ws) == 0 and (buf[16 + need:] == 77).all()
        check(out, c)


def test_windows_and_sinks_past_every_length():
    c = build(8, 2, 2, [300], [20], 16, seed=31)
    h = handle(8, 2, 2)
    want, _ = run(h, c)
    for window, sinks in ((2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (320, 0), (5, 2 ** 31 - 1), (0, 7)):
        out, ws = run(h, c, window, sinks)
        assert status(ws) == 0 and torch.equal(out, want)
    a, _ = run(h, c, 319, 0)
    assert not torch.equal(a, want)


def test_agrees_with_paged_attention():
    c = build(8, 2, 2, [1000, 77], [9, 30], 16, seed=40)
    h = handle(8, 2, 2)
    want, ws2 = h.paged_attention(c["qkv"].cuda(), dev(c["qsl"]), dev(c["lens"]), dev(np.maximum(c["tables"], 0)),
                                  c["ck"].cuda(), c["cv"].cuda(), 30, 1009)
    assert status(ws2) == 0
    check(want, c)
    out, ws = run(h, c)
    assert status(ws) == 0
    check(out, c)


def test_pages_that_no_token_sees_are_not_looked_at():
    # block ids out of range before the window and past the sinks
    for q8 in (False, True):
        c = build(8, 2, 2, [900], [3], 16, seed=41, q8=q8)
        h = handle(8, 2, 2)
        want = run(h, c, 100, 20)[0].clone()
        d = dict(c, tables=c["tables"].copy())
        d["tables"][0, 2:50] = 10 ** 6                     # positions 32 .. 799: sinks are 0 .. 19, the window starts at 801
        out, ws = run(h, d, 100, 20)
        assert status(ws) == 0 and torch.equal(out, want)


def test_bad_pages_and_counts_raise_the_status():
    for q8 in (False, True):
        c = build(8, 2, 2, [40, 20], [3, 2], 16, seed=4, q8=q8)
        h = handle(8, 2, 2)
        for at, v in (((0, 1), 10_000), ((1, 0), -1)):
            d = dict(c, tables=c["tables"].copy())
            d["tables"][at] = v
            out, ws = run(h, d)
            assert status(ws) == tl.TP_ERR_SHAPE and torch.isfinite(out.float()).all()
        for qsl, lens in (([0, 3, 2], c["lens"]), ([0, 3, 6], c["lens"]), ([-1, 3, 5], c["lens"]), (c["qsl"], [2, 22]),
                          (c["qsl"], [43, 1 << 30]), (c["qsl"], [43, -1]), ([0, 2 ** 31 - 1, 5], c["lens"])):
            _, ws = run(h, dict(c, qsl=np.array(qsl), lens=list(lens)), max_q=3, max_len=48)
            assert status(ws) == tl.TP_ERR_SHAPE
        # a request of bad counts does not disturb the others
        out, ws = run(h, dict(c, lens=[1, 22]), max_q=3, max_len=48,
                      out=torch.full((2, 5, 512), 5.0, dtype=torch.bfloat16, device="cuda"))
        assert status(ws) == tl.TP_ERR_SHAPE and (out[:, :3] == 5.0).all()
        good, _ = run(h, c)
        assert torch.equal(out[:, 3:], good[:, 3:])


def test_captured_and_replayed_with_other_lengths():
    for q8 in (False, True):
        h = handle(8, 2, 2)
        c = build(8, 2, 2, [700, 100], [1, 40], 16, seed=70, q8=q8)
        d = build(8, 2, 2, [520, 33], [11, 30], 16, seed=70, q8=q8)    # as many tokens, other lengths and pages
        nb = max(c["ck"].shape[1], d["ck"].shape[1])

        def grown(x, dim, size):
            pad = torch.zeros(*x.shape[:dim], size - x.shape[dim], *x.shape[dim + 1:], dtype=torch.uint8)
            raw = x.view(torch.uint8) if x.dtype is torch.float8_e4m3fn else x
            return torch.cat([raw, pad.to(raw.dtype)], dim).view(x.dtype)
        for x in (c, d):
            for k in ("ck", "cv", "sk", "sv"):
                x[k] = None if x[k] is None else grown(x[k], 1, nb)
            x["tables"] = np.pad(x["tables"], ((0, 0), (0, 50 - x["tables"].shape[1])), constant_values=-1)
        cuda = {k: None if c[k] is None else c[k].cuda() for k in ("qkv", "ck", "cv", "sk", "sv")}
        qsl, lens, tables = dev(c["qsl"]), dev(c["lens"]), dev(c["tables"])
        st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            out, ws = h.chunk_attention(cuda["qkv"], qsl, lens, tables, cuda["ck"], cuda["cv"], 40, 720, 300, 9, cuda["sk"],
                                        cuda["sv"], stream=st)
        for x in (c, d, c):
            qsl.copy_(dev(x["qsl"]))
            lens.copy_(dev(x["lens"]))
            tables.copy_(dev(x["tables"]))
            for k, v in cuda.items():
                if v is not None:
                    (v.view(torch.uint8) if v.dtype is torch.float8_e4m3fn else v).copy_(
                        x[k].view(torch.uint8) if v.dtype is torch.float8_e4m3fn else x[k])
            g.replay()
            assert status(ws) == 0
            check(out, x, 300, 9)


def test_two_calls_at_once_with_workspaces_of_their_own():
    h = handle(8, 2, 2)
    cs = [build(8, 2, 2, [3000, 200], [1, 150], 16, seed=80, q8=False), build(8, 2, 2, [2500, 900], [3, 1], 16, seed=81, q8=True)]
    outs, wss, sts = [], [], [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, st in zip(cs, sts):
            out, ws = run(h, c, 800, 3, stream=st)
            outs.append((c, out))
            wss.append(ws)
    torch.cuda.synchronize()
    assert all(status(w) == 0 for w in wss)
    for c, out in outs[:2]:
        check(out, c, 800, 3)
    for k, (c, out) in enumerate(outs[2:]):
        assert torch.equal(out, outs[k % 2][1])


def test_wait_limit_runs_out_and_context_survives():
    # in the kernel of 128-row tiles, whose walking warp is four items of some 100 us ahead and waits for a place;
    # no wait of the kernel for up to 16 rows lasts longer than the first suspended try
    for q8 in (False, True):
        reqs, ctx, n = 110, 8192, 20
        c = build(8, 8, 1, [ctx], [n], 16, seed=60, q8=q8)
        h = handle(8, 8, 1)
        many = dict(c, tables=np.repeat(c["tables"], reqs, 0), lens=[ctx + n] * reqs, qsl=np.arange(reqs + 1) * n,
                    n=[n] * reqs, T=reqs * n, qkv=c["qkv"].repeat(1, reqs, 1))
        good, ws = run(h, many)
        good = good.clone()
        assert status(ws) == 0
        tl.set_wait_timeout(1)                              # waits of more than one suspended try (20 us) run out
        try:
            _, ws = run(h, many, ws=ws)
            st = status(ws)                                 # returns: nothing hung, nothing faulted
        finally:
            tl.set_wait_timeout(2_000_000_000)
        assert st == tl.TP_ERR_TIMEOUT
        ws.zero_()
        out, ws = run(h, many, ws=ws)
        assert status(ws) == 0 and torch.equal(out, good)


def test_refusals():
    h, h64, L = handle(8, 2, 2), handle(8, 2, 2, hd=64), tl.lib()
    n = ctypes.c_int64()

    def at(x):
        return None if x is None else ctypes.c_void_p(x)

    def call(hd=h.handle, T=8, q=1 << 24, qsl=1 << 16, lens=1 << 17, reqs=2, mq=4, ml=64, bt=1 << 18, mb=4, window=0, sinks=0,
             ck=1 << 25, cv=1 << 26, sk=None, sv=None, nb=8, bs=16, out=1 << 27, ws=1 << 40, wb=1 << 40):
        return L.tp_chunk_attention(hd, T, at(q), at(qsl), at(lens), reqs, mq, ml, at(bt), mb, window, sinks, at(ck), at(cv),
                                    at(sk), at(sv), nb, bs, at(out), at(ws), wb, None)
    assert call(T=0) == tl.TP_OK
    assert call(hd=None) == tl.TP_ERR_ARG and call(hd=h64.handle) == tl.TP_ERR_UNSUPPORTED and call(T=-1) == tl.TP_ERR_SHAPE
    assert call(reqs=0) == tl.TP_ERR_SHAPE and call(mq=0) == tl.TP_ERR_SHAPE and call(ml=3) == tl.TP_ERR_SHAPE
    assert call(nb=0) == tl.TP_ERR_SHAPE and call(bs=0) == tl.TP_ERR_SHAPE and call(mb=3) == tl.TP_ERR_SHAPE
    assert call(nb=1 << 31) == tl.TP_ERR_UNSUPPORTED and call(nb=1 << 27) == tl.TP_ERR_UNSUPPORTED
    assert call(ml=(1 << 26) + 1, mb=1 << 23) == tl.TP_ERR_UNSUPPORTED
    assert call(window=-1) == tl.TP_ERR_ARG and call(sinks=-1) == tl.TP_ERR_ARG
    assert call(sk=1 << 28) == tl.TP_ERR_ARG and call(sv=1 << 28) == tl.TP_ERR_ARG
    for k in ("q", "ck", "cv", "out", "ws"):
        assert call(**{k: None}) == tl.TP_ERR_ARG and call(**{k: (1 << 30) + 8}) == tl.TP_ERR_ARG
    for k in ("qsl", "lens", "bt"):
        assert call(**{k: None}) == tl.TP_ERR_ARG and call(**{k: (1 << 16) + 2}) == tl.TP_ERR_ARG
    assert call(wb=16) == tl.TP_ERR_ARG and b"too small" in L.tp_last_error()
    for out in (1 << 24, (1 << 24) + 256, 1 << 25, 1 << 26, 1 << 16, 1 << 18):
        assert call(out=out) == tl.TP_ERR_ARG and b"overlaps" in L.tp_last_error()
    wide = tl.make_config(tl.TP_BLOCK_ATTN_PROJ, 1, 64, n_q_heads=257, n_kv_heads=1, head_dim=128)
    z = torch.zeros(257 * 128, 64, dtype=torch.bfloat16, device="cuda")
    hw = tl.TPLinear(wide, [z, z[:128].contiguous(), z[:128].contiguous(), z.t().contiguous()])
    assert call(hd=hw.handle) == tl.TP_ERR_UNSUPPORTED
    f = L.tp_chunk_attention_workspace_size
    assert f(h.handle, 0, 1, 1, ctypes.byref(n)) == tl.TP_ERR_SHAPE and f(h.handle, 1, 1, 1, None) == tl.TP_ERR_ARG
    assert f(None, 1, 1, 1, ctypes.byref(n)) == tl.TP_ERR_ARG
    assert f(h.handle, 1, 1, (1 << 26) + 1, ctypes.byref(n)) == tl.TP_ERR_UNSUPPORTED
    assert f(h.handle, 1, 1 << 24, 1 << 26, ctypes.byref(n)) == tl.TP_OK
    c = build(8, 2, 2, [20], [3], 16, seed=1, q8=True)
    with pytest.raises(ValueError):
        run(h, dict(c, sv=None))
    with pytest.raises(ValueError):
        run(h, dict(c, sk=None, sv=None))
    with pytest.raises(ValueError):
        run(h, dict(c, sk=c["sk"][:, :1]))
    with pytest.raises(ValueError):
        run(h, dict(c, tables=c["tables"][0]))
