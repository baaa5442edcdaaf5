"""Token-tree masks and attention on the GPU (tp_tree_mask, tp_tree_attention) against the float64 oracle.

Masks and positions are whole numbers: equal. Attention, element by element, with A = the same
weighted mean over |v| (sum p |v| / sum p, from the oracle): rounding P to bf16 moves a weight by
at most 2^-8 of itself (and the sum of weights with it, by no more), so the mean by 2^-7 A; fp32
scores of |q . k| summed over 128 products, scaled, are off by under 2^-10 of a weight for the
|q . k| <= 500 here (128 * 2^-24 * 500 / sqrt(128) = 2^-11.4, and as much again for the exponential);
the output's rounding is 2^-8 |ref|. So |got - ref| <= 2^-8 |ref| + (2^-7 + 2^-10) A.
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import workloads
import tensor_linear_layers_gb300 as tl

pytestmark = pytest.mark.gpu
f64 = oracle.bf16_to_f64


@pytest.fixture(scope="module", autouse=True)
def built():
    from tensor_linear_layers_gb300 import _build
    _build.build()
    tl.lib()
    torch.cuda.set_device(0)


def handle(nq, nkv, t, flags=0, hd=128, H=64):
    cfg = tl.make_config(tl.TP_BLOCK_ATTN_PROJ, t, H, n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, flags=flags)
    z = torch.zeros(nq * hd, H, dtype=torch.bfloat16, device="cuda")
    return tl.TPLinear(cfg, [z, z[:nkv * hd].contiguous(), z[:nkv * hd].contiguous(), z.t().contiguous()])


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def status(ws):
    torch.cuda.synchronize()
    return int(ws[:4].view(torch.int32))


def random_parents(rng, n, back=4):
    return [max(-1, i - int(rng.integers(1, back + 1))) for i in range(n)]


def build(nq, nkv, t, ctx, n, bs, seed, pad=0, extra_blocks=3, scale=1.0):
    """Inputs of requests with ctx[b] cached and n[b] drafted tokens on scattered pages."""
    rng = np.random.default_rng(seed)
    lens = [c + k for c, k in zip(ctx, n)]
    need = [-(-k // bs) for k in lens]
    nb = sum(need) + extra_blocks
    perm = rng.permutation(nb)
    tables = np.full((len(lens), max(max(need), 1) + 1), -5, dtype=np.int32)     # entries past a request are not read
    used = 0
    for b, k in enumerate(need):
        tables[b, :k] = perm[used:used + k]
        used += k
    kv_per = 1 if t >= nkv else nkv // t
    T = sum(n) + pad
    qkv = workloads.draw((t, max(T, 1), (nq // t + 2 * kv_per) * 128), seed, 0)[:, :T]
    if scale != 1.0:
        qkv = (qkv.float() * scale).to(torch.bfloat16)
    ck = workloads.draw((t, nb, bs, kv_per, 128), seed, 1)
    cv = workloads.draw((t, nb, bs, kv_per, 128), seed, 2)
    parents = [random_parents(rng, k) for k in n]
    return dict(lens=lens, tables=tables, qkv=qkv.contiguous(), ck=ck, cv=cv, parents=parents,
                qsl=np.concatenate([[0], np.cumsum(n)]), n=n, T=T, bs=bs)


def run(h, c, mask=None, out=None, max_q=None, max_len=None, ws=None):
    mq = max(max(c["n"]), 1) if max_q is None else max_q
    ml = max(c["lens"] + [mq]) if max_len is None else max_len
    if mask is None:
        flat = sum(c["parents"], []) + [-1] * (c["T"] - sum(c["n"]))
        mask, _, mws = tl.tree_mask(dev(flat), dev(c["qsl"]), dev(c["lens"]), mq)
        assert status(mws) == 0
    return h.tree_attention(c["qkv"].cuda(), dev(c["qsl"]), dev(c["lens"]), dev(c["tables"]), mask, c["ck"].cuda(),
                            c["cv"].cuda(), mq, ml, out=out, ws=ws)


def check(got, c, nq, nkv, t, sees=None, rows=None):
    sees = [oracle.tree_sees(p) if p else np.zeros((0, 0), bool) for p in c["parents"]] if sees is None else sees
    a = (c["qkv"], c["qsl"], c["lens"], c["tables"], sees, c["ck"])
    ref = oracle.tree_attention(*a, c["cv"], nq, nkv, 128, t, c["bs"])
    mean = oracle.tree_attention(*a, c["cv"].abs(), nq, nkv, 128, t, c["bs"])
    g = f64(got.cpu())
    used = slice(0, sum(c["n"]))
    err = np.abs(g - ref)[:, used]
    tol = (2.0 ** -8 * np.abs(ref) + (2.0 ** -7 + 2.0 ** -10) * mean)[:, used]
    assert (err <= tol).all(), float((err - tol).max())


# ------------------------------------------------------------------ masks and positions
@pytest.mark.parametrize("n", [[1], [5, 0, 33], [64, 1, 7], [256, 255], [32, 31]])
def test_tree_mask_equals_the_oracles(n):
    rng = np.random.default_rng(len(n) + n[0])
    parents = [random_parents(rng, k, 9) for k in n]
    ctx = [int(x) for x in rng.integers(0, 5000, len(n))]
    words = -(-max(n) // 32)
    flat = dev(sum(parents, []) + [-1, -1])                             # two rows of no request
    mask = torch.full((len(flat), words), 77, dtype=torch.int32, device="cuda")
    pos = torch.full((len(flat),), 77, dtype=torch.int32, device="cuda")
    _, _, ws = tl.tree_mask(flat, dev(np.concatenate([[0], np.cumsum(n)])), dev([c + k for c, k in zip(ctx, n)]),
                            max(n), out=(mask, pos))
    assert status(ws) == 0
    at = 0
    for p, c in zip(parents, ctx):
        sees = oracle.tree_sees(p)
        np.testing.assert_array_equal(mask[at:at + len(p)].cpu().numpy(), oracle.mask_words(sees, words))
        np.testing.assert_array_equal(pos[at:at + len(p)].cpu().numpy(), c + sees.sum(1) - 1)
        at += len(p)
    assert (mask[at:] == 77).all() and (pos[at:] == 77).all()


def test_tree_mask_bad_parents_and_counts():
    parents = dev([-1, 1, 0, 2, 7, -1, -2, 0, -1])
    qsl, lens = dev([0, 5, 7, 9]), dev([9, 4, 1])                       # the last request has 2 drafts but 1 token
    mask, pos, ws = tl.tree_mask(parents, qsl, lens, 8, out=(torch.full((9, 1), 77, dtype=torch.int32, device="cuda"),
                                                             torch.full((9,), 77, dtype=torch.int32, device="cuda")))
    assert status(ws) == tl.TP_ERR_SHAPE
    # token 1 is its own parent, token 4's comes after it, token 6's is below -1: empty rows, position -1
    assert mask[:, 0].tolist() == [1, 0, 5, 13, 0, 1, 0, 77, 77]
    assert pos.tolist() == [4, -1, 5, 6, -1, 2, -1, 77, 77]
    for bad in ([0, 5, 4, 9], [0, 5, 7, 10], [-1, 5, 7, 9], [0, 9, 9, 9]):
        _, _, ws = tl.tree_mask(parents, dev(bad), dev([20, 20, 20]), 8)
        assert status(ws) == tl.TP_ERR_SHAPE


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("nq,nkv,t,ctx,n,bs", [
    (8, 2, 2, [0], [1], 16),                              # the shortest: one token that sees itself
    (8, 2, 2, [1, 37, 300, 129], [1, 1, 1, 1], 16),       # decode: one drafted token each
    (8, 2, 4, [200, 64], [5, 9], 8),                      # t > nkv: kv heads replicated
    (4, 4, 2, [90, 0, 400], [5, 17, 3], 16),              # a request without cached tokens
    (16, 2, 1, [700], [20], 32),                          # groups of 8 q heads, more rows than one tile
    (8, 1, 1, [131], [40], 24),                           # blocks of 24: pages end inside tiles; two tiles of rows
    (8, 4, 8, [129, 40], [3, 1], 1),                      # blocks of one token
    (28, 4, 4, [255, 256, 257, 128, 127], [7, 8, 1, 2, 3], 64),   # groups of 7; lengths around tile edges
    (4, 4, 1, [500], [64], 128),                          # one q head per kv head
    (8, 1, 2, [260], [70], 5),                            # 280 rows a shard: three tiles of rows
    (8, 2, 2, [50, 60], [0, 4], 16),                      # a request without drafted tokens
    (64, 1, 1, [100, 260], [5, 3], 16),                   # one kv head for 64 q heads
])
@pytest.mark.parametrize("gathered", [False, True])
def test_tree_attention_matches_oracle(nq, nkv, t, ctx, n, bs, gathered):
    c = build(nq, nkv, t, ctx, n, bs, seed=len(n) * 10 + t)
    h = handle(nq, nkv, t, tl.TP_FLAG_GATHERED if gathered else 0)
    if gathered:
        cg = dict(c, qkv=c["qkv"].permute(1, 0, 2).reshape(c["T"], -1).contiguous())
        out, ws = run(h, cg)
        out = out.view(c["T"], t, -1).permute(1, 0, 2)
    else:
        out, ws = run(h, c)
    assert status(ws) == 0
    check(out, c, nq, nkv, t)


def test_masks_that_are_not_trees_and_empty_rows():
    nq, nkv, t = 8, 2, 2
    rng = np.random.default_rng(3)
    c = build(nq, nkv, t, [0, 150], [40, 35], 16, seed=3)
    sees = [rng.random((k, k)) < 0.3 for k in c["n"]]
    sees[0][[0, 17, 39]] = False                          # nothing cached and nothing drafted: rows of zeros
    sees[1][4] = False
    mask = torch.cat([torch.from_numpy(oracle.mask_words(s, 3)) for s in sees]).cuda()
    mask[:, 1] |= torch.where(torch.arange(75, device="cuda") < 40, -256, -8).int()     # bits past the drafts: not read
    mask[:, 2] = -1
    out, ws = run(handle(nq, nkv, t), c, mask=mask, max_q=70)
    assert status(ws) == 0
    assert (out[:, [0, 17, 39]] == 0).all()
    check(out, c, nq, nkv, t, sees)


def test_rows_of_no_request_are_left_as_they_were():
    c = build(8, 2, 2, [100, 30], [6, 3], 16, seed=8, pad=5)
    out = torch.full((2, 14, 512), 5.0, dtype=torch.bfloat16, device="cuda")
    _, ws = run(handle(8, 2, 2), c, out=out)
    assert status(ws) == 0 and (out[:, 9:] == 5.0).all()
    check(out, c, 8, 2, 2)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_a_token_does_not_see_has_no_effect(bad):
    # NaN and infinities in k and v of one branch, and in the rest of the pages, which nobody sees
    nq, nkv, t, bs = 8, 2, 2, 16
    c = build(nq, nkv, t, [120, 5], [30, 9], bs, seed=12)
    c["parents"] = [random_parents(np.random.default_rng(1), 30), [-1, 0, 0, 1, 2, -1, 5, 3, 4]]
    h = handle(nq, nkv, t)
    clean, _ = run(h, c)
    clean = clean.clone()
    sees = [oracle.tree_sees(p) for p in c["parents"]]
    ck, cv = c["ck"].clone(), c["cv"].clone()
    tainted = np.zeros(39, dtype=bool)
    for b, j, q0, ctx in ((0, 11, 0, 120), (1, 2, 30, 5)):
        s = oracle.slot_of(c["tables"], b, ctx + j, bs)
        ck[:, s // bs, s % bs] = bad
        cv[:, s // bs, s % bs, :, 1::2] = bad
        tainted[q0:q0 + c["n"][b]] |= sees[b][:, j]
    for b, L in enumerate(c["lens"]):                     # the last page past the request's tokens
        if L % bs:
            ck[:, c["tables"][b, L // bs], L % bs:] = bad
            cv[:, c["tables"][b, L // bs], L % bs:] = bad
    d = dict(c, ck=ck, cv=cv)
    got, ws = run(h, d)
    assert status(ws) == 0
    assert torch.equal(got[:, ~tainted], clean[:, ~tainted])
    assert not torch.isfinite(got[:, tainted].float()).all(-1).any()
    # bad values in v alone reach the tokens that see them, in their own dimensions
    got, _ = run(h, dict(c, cv=cv))
    g = got.float().cpu().view(2, 39, 4, 64, 2)
    assert torch.equal(got[:, ~tainted], clean[:, ~tainted])
    assert not torch.isfinite(g[:, tainted][..., 1]).any()
    assert torch.isfinite(g[:, tainted][..., 0]).all()


def test_large_scores_and_equal_bits_on_repetition():
    # peaked softmax (scores of some hundreds) and the same call again: the same bits
    nq, nkv, t = 16, 4, 2
    c = build(nq, nkv, t, [1500, 70, 900], [12, 30, 1], 16, seed=21, scale=4.0)
    h = handle(nq, nkv, t)
    ws = torch.zeros(h.tree_attention_workspace_size(3, 30, 1512), dtype=torch.uint8, device="cuda")
    a, _ = run(h, c, ws=ws)
    a = a.clone()
    check(a, c, nq, nkv, t)
    for _ in range(3):
        b, _ = run(h, c, ws=ws)
        assert torch.equal(a, b)
    assert status(ws) == 0


def test_workspace_on_a_16_byte_boundary_and_odd_row_counts():
    # partial slots of 18, 5 and 27 rows, the workspace aligned to 16 bytes only, and nothing written past it
    for nq, nkv, t, n in ((8, 2, 4, 9), (4, 4, 2, 5), (9, 3, 1, 9)):
        c = build(nq, nkv, t, [700, 64], [n, 2], 16, seed=n)
        h = handle(nq, nkv, t)
        need = h.tree_attention_workspace_size(2, n, 700 + n)
        buf = torch.zeros(need + 64, dtype=torch.uint8, device="cuda")
        buf[16 + need:] = 77
        out, ws = run(h, c, ws=buf[16:16 + need])
        assert status(ws) == 0
        assert (buf[16 + need:] == 77).all()
        check(out, c, nq, nkv, t)


def test_long_context_many_requests():
    # more work than one pass of the GPU: splits that start and end inside requests
    nq, nkv, t = 8, 2, 2
    rng = np.random.default_rng(5)
    n = [int(x) for x in rng.integers(1, 9, 40)]
    ctx = [int(x) for x in rng.integers(0, 900, 40)]
    ctx[3], n[3] = 6000, 8
    c = build(nq, nkv, t, ctx, n, 16, seed=33)
    out, ws = run(handle(nq, nkv, t), c)
    assert status(ws) == 0
    check(out, c, nq, nkv, t)


def test_more_requests_than_one_batch_and_long_runs_of_empty_ones():
    # 300 requests, most of them without drafted tokens (a padded batch), work at both ends and between
    nq, nkv, t = 4, 2, 1
    n, ctx = [0] * 300, [0] * 300
    rng = np.random.default_rng(9)
    for b in (0, 31, 32, 127, 128, 200, 299):
        n[b], ctx[b] = int(rng.integers(1, 6)), int(rng.integers(0, 400))
    for b in range(250, 298):
        ctx[b] = 17                                         # cached tokens, nothing drafted
    c = build(nq, nkv, t, ctx, n, 16, seed=50)
    out, ws = run(handle(nq, nkv, t), c)
    assert status(ws) == 0
    check(out, c, nq, nkv, t)
    # nobody has a drafted token: nothing is computed, nothing written
    d = dict(c, qsl=np.zeros(301, dtype=np.int64), lens=ctx)
    keep = torch.full_like(out, 5.0)
    mask = torch.zeros(c["T"], 1, dtype=torch.int32, device="cuda")
    _, ws = run(handle(nq, nkv, t), d, mask=mask, out=keep, max_q=5, max_len=max(c["lens"]))
    assert status(ws) == 0 and (keep == 5.0).all()


def test_wait_limit_runs_out_and_context_survives():
    # 24 requests that share one document's pages (read only): some 100 us of work for every SM, in which
    # the warp that looks at the drafted tokens' values waits for the last chunk of its item
    nq = nkv = 8
    reqs, ctx, n = 24, 8192, 2
    c = build(nq, nkv, 1, [ctx], [n], 16, seed=60)
    h = handle(nq, nkv, 1)
    many = dict(c, tables=np.repeat(c["tables"], reqs, 0), lens=[ctx + n] * reqs, qsl=np.arange(reqs + 1) * n,
                n=[n] * reqs, T=reqs * n, qkv=c["qkv"].repeat(1, reqs, 1), parents=c["parents"] * reqs)
    good, ws = run(h, many)
    good = good.clone()
    assert status(ws) == 0
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
    # requests 0 and 17 against the oracle
    ref = oracle.tree_attention(c["qkv"], [0, n], [ctx + n], c["tables"], [oracle.tree_sees(c["parents"][0])], c["ck"],
                                c["cv"], nq, nkv, 128, 1, 16)
    for b in (0, 17):
        g = f64(out[:, b * n:(b + 1) * n].cpu())
        assert np.abs(g - ref).max() <= 2e-2 * np.abs(ref).max()


def test_chain_agrees_with_paged_attention():
    # a chain of drafted tokens is the causal case that tp_paged_attention computes
    nq, nkv, t = 8, 2, 2
    c = build(nq, nkv, t, [1000, 77], [9, 30], 16, seed=40)
    c["parents"] = [list(range(-1, k - 1)) for k in c["n"]]
    h = handle(nq, nkv, t)
    out, ws = run(h, c)
    want, ws2 = h.paged_attention(c["qkv"].cuda(), dev(c["qsl"]), dev(c["lens"]), dev(np.maximum(c["tables"], 0)),
                                  c["ck"].cuda(), c["cv"].cuda(), 30, 1009)
    assert status(ws) == 0 and status(ws2) == 0
    check(out, c, nq, nkv, t)
    check(want, c, nq, nkv, t)


def test_bad_pages_and_counts_raise_the_status():
    nq, nkv, t, bs = 8, 2, 2, 16
    c = build(nq, nkv, t, [40, 20], [3, 2], bs, seed=4)
    h = handle(nq, nkv, t)
    for change in (lambda x: x["tables"].__setitem__((0, 1), 10_000), lambda x: x["tables"].__setitem__((1, 0), -1)):
        d = dict(c, tables=c["tables"].copy())
        change(d)
        out, ws = run(h, d)
        assert status(ws) == tl.TP_ERR_SHAPE and torch.isfinite(out.float()).all()
    mask, _, _ = tl.tree_mask(dev(sum(c["parents"], [])), dev(c["qsl"]), dev(c["lens"]), 3)
    for qsl, lens in (([0, 3, 2], c["lens"]), ([0, 3, 6], c["lens"]), ([-1, 3, 5], c["lens"]), (c["qsl"], [2, 22]),
                      (c["qsl"], [43, 1 << 30])):
        d = dict(c, qsl=np.array(qsl), lens=list(lens))
        _, ws = run(h, d, mask=mask, max_q=3, max_len=48)
        assert status(ws) == tl.TP_ERR_SHAPE
    # a request of bad counts does not disturb the others
    out, ws = run(h, dict(c, lens=[1, 22]), mask=mask, max_q=3, max_len=48,
                  out=torch.full((2, 5, 512), 5.0, dtype=torch.bfloat16, device="cuda"))
    assert status(ws) == tl.TP_ERR_SHAPE and (out[:, :3] == 5.0).all()
    good, _ = run(h, c)
    assert torch.equal(out[:, 3:], good[:, 3:])


def test_refusals():
    h, h64 = handle(8, 2, 2), handle(8, 2, 2, hd=64)
    L, p = tl.lib(), ctypes.c_void_p(0x10000)
    n = ctypes.c_int64()

    def call(hd=h.handle, T=8, q=p, qsl=p, lens=p, reqs=2, mq=4, ml=64, bt=p, mb=4, mask=p, words=1, ck=p, cv=p, nb=8, bs=16,
             out=p, ws=p, wb=1 << 40):
        return L.tp_tree_attention(hd, T, q, qsl, lens, reqs, mq, ml, bt, mb, mask, words, ck, cv, nb, bs, out, ws, wb, None)
    odd4, odd16 = ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10008)
    assert call(T=0) == tl.TP_OK
    assert call(hd=h64.handle) == tl.TP_ERR_UNSUPPORTED and call(T=-1) == tl.TP_ERR_SHAPE
    assert call(reqs=0) == tl.TP_ERR_SHAPE and call(mq=0) == tl.TP_ERR_SHAPE and call(ml=3) == tl.TP_ERR_SHAPE
    assert call(mq=257, ml=300, words=9, mb=40) == tl.TP_ERR_UNSUPPORTED
    assert call(words=0) == tl.TP_ERR_SHAPE and call(mq=40, ml=64) == tl.TP_ERR_SHAPE
    assert call(nb=0) == tl.TP_ERR_SHAPE and call(bs=0) == tl.TP_ERR_SHAPE and call(mb=3) == tl.TP_ERR_SHAPE
    assert call(nb=1 << 31) == tl.TP_ERR_UNSUPPORTED and call(nb=1 << 27) == tl.TP_ERR_UNSUPPORTED
    for k in ("q", "ck", "cv", "out", "ws"):
        assert call(**{k: None}) == tl.TP_ERR_ARG and call(**{k: odd16}) == tl.TP_ERR_ARG
    for k in ("qsl", "lens", "bt", "mask"):
        assert call(**{k: None}) == tl.TP_ERR_ARG and call(**{k: odd4}) == tl.TP_ERR_ARG
    assert call(wb=16) == tl.TP_ERR_ARG and b"too small" in L.tp_last_error()
    assert L.tp_tree_attention_workspace_size(h.handle, 0, 1, 1, ctypes.byref(n)) == tl.TP_ERR_SHAPE
    assert L.tp_tree_attention_workspace_size(h.handle, 1, 1, 1, None) == tl.TP_ERR_ARG
    c = build(8, 2, 2, [20], [3], 16, seed=1)
    with pytest.raises(TypeError):
        run(h, c, mask=torch.zeros(3, 1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        run(h, c, mask=torch.zeros(2, 1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        run(h, dict(c, ck=c["ck"][:, :, :, :, :64]))


def test_refusals_of_outputs_over_inputs_and_of_long_requests():
    h, L, n = handle(8, 2, 2), tl.lib(), ctypes.c_int64()

    def at(x):
        return ctypes.c_void_p(x)
    p, ws_bytes = at(0x10000), 1 << 40
    width = h.kv_cache_shape(1, 1)[0] * 8 * (4 + 2) * 128 * 2    # an upper bound on the bytes of 8 rows of qkv

    def attention(out, ml=64, mb=4, bs=16):
        return L.tp_tree_attention(h.handle, 8, at(1 << 24), p, p, 2, 4, ml, p, mb, p, 1, p, p, 8, bs, at(out), p, ws_bytes,
                                   None)
    for out in (1 << 24, (1 << 24) + 256, (1 << 24) - 256):
        assert width > 256 and attention(out) == tl.TP_ERR_ARG and b"overlaps" in L.tp_last_error()
    long = (1 << 26) + 1
    assert attention(1 << 20, ml=long, mb=1 << 23) == tl.TP_ERR_UNSUPPORTED
    assert L.tp_tree_attention_workspace_size(h.handle, 1, 1, long, ctypes.byref(n)) == tl.TP_ERR_UNSUPPORTED
    assert L.tp_tree_attention_workspace_size(h.handle, 1, 1, long - 1, ctypes.byref(n)) == tl.TP_OK

    def mask(parents=0x10000, qsl=0x20000, lens=0x30000, out=0x40000, pos=0x50000):
        return L.tp_tree_mask(8, 2, 4, at(parents), at(qsl), at(lens), at(out), 1, at(pos), at(0x60000), 16, None)
    for k, v in (("out", 0x10000), ("out", 0x20008), ("out", 0x30004), ("pos", 0x10004), ("pos", 0x20008),
                 ("pos", 0x2fffc), ("pos", 0x40010)):
        assert mask(**{k: v}) == tl.TP_ERR_ARG and b"overlaps" in L.tp_last_error()
