"""Rotary positions and per-head norms on the GPU (tp_rope_table, tp_qk_norm_rope) against the float64 oracle.

Tolerance. One rounding to bf16 is off by at most 2^-8 of the value (half a step). Before it, in
fp32: the table's cos and sin are off by 2^-24 of themselves, the norm's factor by less than
(hd / 2 + 4) 2^-24 <= 2^-16 (a sum of hd <= 256 squares), the rotation adds three roundings of
terms no larger than 2 max|x'| m: together under 2^-14 max|x'| m of the head. So
|got - ref| <= 2^-8 |ref| + 2^-14 m max|x'|. v and padding rows are copies: exact. The cache
holds the bits of the output.
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


def handle(nq, nkv, hd, t, flags=0, H=64):
    cfg = tl.make_config(tl.TP_BLOCK_ATTN_PROJ, t, H, n_q_heads=nq, n_kv_heads=nkv, head_dim=hd, flags=flags)
    z = torch.zeros(nq * hd, H, dtype=torch.bfloat16, device="cuda")
    return tl.TPLinear(cfg, [z, z[:nkv * hd].contiguous(), z[:nkv * hd].contiguous(), z.t().contiguous()])


def width(nq, nkv, hd, t):
    return (nq // t + 2 * (1 if t >= nkv else nkv // t)) * hd


def gamma(hd, i):
    return workloads.draw((hd,), 90, i, kind="uniform", a=0.5, b=1.5)


def heads_of(a, nq, nkv, hd, t):
    """[t, T, heads, hd] view of a shard-major qkv."""
    return a.reshape(t, a.shape[1], -1, hd)


def check(got, qkv, pos, nq, nkv, hd, t, rd, kw, inter, gq, gk, eps):
    """Elementwise bound of the module docstring; returns the reference."""
    f, m = oracle.rope_frequencies(rd, kw["base"], kw.get("scaling", "none"), kw.get("factor", 1.0),
                                   kw.get("original_max_position", 0))
    m = kw.get("attn_factor", 0.0) or m
    ref = oracle.qk_norm_rope(qkv, pos, f, nq, nkv, hd, t, inter, m, gq, gk, eps)
    flat = oracle.qk_norm_rope(qkv, pos, 0 * f, nq, nkv, hd, t, inter, 1.0, gq, gk, eps)     # x' alone
    big = np.abs(heads_of(flat, nq, nkv, hd, t)).max(-1, keepdims=True)
    tol = 2.0 ** -8 * np.abs(heads_of(ref, nq, nkv, hd, t)) + 2.0 ** -14 * max(m, 1.0) * big
    q_per = nq // t
    kv_per = 1 if t >= nkv else nkv // t
    tol[:, :, q_per + kv_per:] = 0                                                           # v: a copy
    err = np.abs(heads_of(f64(got.cpu()), nq, nkv, hd, t) - heads_of(ref, nq, nkv, hd, t))
    assert (err <= tol).all(), float((err - tol).max())
    return ref


CASES = [  # nq, nkv, hd, t, T, rd, interleaved, q gamma, k gamma, rope arguments
    (8, 2, 128, 2, 33, 128, False, False, False, dict(base=10000.0)),
    (8, 2, 128, 4, 5, 128, True, True, True, dict(base=500000.0, scaling="bands", factor=8.0, original_max_position=8192)),
    (28, 4, 128, 4, 70, 64, False, True, True, dict(base=1e6, scaling="yarn", factor=4.0, original_max_position=32768)),
    (4, 4, 128, 1, 1, 32, True, True, False, dict(base=10000.0, scaling="linear", factor=2.0)),
    (4, 2, 128, 2, 9, 20, False, False, True, dict(base=10000.0, scaling="ntk", factor=4.0)),
    (4, 2, 128, 8 // 4, 300, 2, True, False, False, dict(base=10000.0)),
    (4, 4, 128, 2, 17, 96, False, True, True, dict(base=10000.0, attn_factor=1.5)),
    (6, 3, 64, 1, 13, 64, False, True, True, dict(base=10000.0)),
    (6, 3, 64, 1, 13, 16, True, True, True, dict(base=10000.0)),
    (4, 2, 96, 1, 21, 24, False, False, False, dict(base=10000.0)),
    (4, 2, 80, 2, 11, 80, True, True, True, dict(base=10000.0)),
    (4, 2, 72, 2, 11, 36, False, True, True, dict(base=10000.0)),
    (2, 1, 8, 1, 4, 8, False, True, True, dict(base=10000.0)),
    (2, 1, 256, 1, 7, 256, False, True, True, dict(base=10000.0)),
    (2, 1, 256, 1, 7, 130, False, True, True, dict(base=10000.0)),
    (2, 1, 256, 1, 7, 64, True, False, True, dict(base=10000.0)),
]


@pytest.mark.parametrize("nq,nkv,hd,t,T,rd,inter,gq,gk,kw", CASES)
@pytest.mark.parametrize("gathered", [False, True])
def test_matches_oracle(nq, nkv, hd, t, T, rd, inter, gq, gk, kw, gathered):
    n_pos = 70000
    h = handle(nq, nkv, hd, t, tl.TP_FLAG_GATHERED if gathered else 0)
    g_q, g_k = gamma(hd, 0) if gq else None, gamma(hd, 1) if gk else None
    r = tl.Rope(n_pos, rd, layout=tl.TP_ROPE_INTERLEAVED if inter else tl.TP_ROPE_HALF, eps=1e-5,
                q_gamma=None if g_q is None else g_q.cuda(), k_gamma=None if g_k is None else g_k.cuda(), **kw)
    qkv = workloads.draw((t, T, width(nq, nkv, hd, t)), 7 * T + rd, 0)
    pos = np.random.default_rng(T).integers(0, n_pos, T)
    pos[0] = 0
    pos[-1] = n_pos - 1
    if T > 3:
        pos[2] = -1                                                  # padding
    posd = torch.from_numpy(pos.astype(np.int32)).cuda()
    src = qkv.cuda()
    if gathered:
        src = src.permute(1, 0, 2).reshape(T, -1).contiguous()
    keep = torch.full_like(src, 7.0)
    out, ws = h.qk_norm_rope(src, posd, r, out=keep)
    inplace, ws2 = h.qk_norm_rope(src.clone(), posd, r, out=None)
    again = src.clone()
    h.qk_norm_rope(again, posd, r, out=again)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32)) == 0 and int(ws2[:4].view(torch.int32)) == 0
    live = torch.from_numpy(pos >= 0)
    rows = (lambda x: x.reshape(T, t, -1).permute(1, 0, 2)) if gathered else (lambda x: x)
    got = rows(out).cpu()
    assert (got[:, ~live] == 7.0).all()                              # a padding row is left as it was
    assert torch.equal(rows(again).cpu()[:, ~live], qkv[:, ~live])
    assert torch.equal(rows(again).cpu()[:, live], got[:, live])     # in place: the same bits
    assert torch.equal(rows(inplace).cpu()[:, live], got[:, live])
    fixed = got.clone()
    fixed[:, ~live] = qkv[:, ~live]
    check(fixed, qkv, pos, nq, nkv, hd, t, rd, kw, inter, g_q, g_k, 1e-5)


def test_far_positions_and_table_bits():
    # the angle of pair 0 at position 1048575 is 1048575 radians: its cosine needs 64 bits before the rounding
    r = tl.Rope(1 << 20, 32, 10000.0, scaling="yarn", factor=16.0, original_max_position=4096)
    torch.cuda.synchronize()
    f, m = oracle.rope_frequencies(32, 10000.0, "yarn", 16.0, 4096)
    pos = np.array([0, 1, 4095, 99991, 1048575])
    ang = pos[:, None] * f[None]
    got = r.table[torch.from_numpy(pos).cuda()].double().cpu().numpy()
    # fp32 rounding (2^-24 of a value up to m) and the 64-bit angle's own 2^-53 * 2^20 rad = 2^-33
    np.testing.assert_allclose(got[:, :16], np.cos(ang) * m, atol=m * (2.0 ** -24 + 2.0 ** -32), rtol=0)
    np.testing.assert_allclose(got[:, 16:], np.sin(ang) * m, atol=m * (2.0 ** -24 + 2.0 ** -32), rtol=0)


@pytest.mark.parametrize("nq,nkv,t,T,bs,rd,inter", [(8, 2, 2, 50, 16, 128, False), (8, 2, 4, 7, 1, 64, True),
                                                    (4, 4, 1, 30, 24, 20, False), (4, 2, 8 // 4, 257, 32, 128, True)])
def test_cache_write_has_the_output_bits(nq, nkv, t, T, bs, rd, inter):
    h = handle(nq, nkv, 128, t)
    r = tl.Rope(4096, rd, layout=int(inter), q_gamma=gamma(128, 0).cuda(), k_gamma=gamma(128, 1).cuda())
    qkv = workloads.draw((t, T, width(nq, nkv, 128, t)), T, 0).cuda()
    nb = -(-T // bs) + 3
    rng = np.random.default_rng(T)
    slots = rng.permutation(nb * bs)[:T].astype(np.int32)
    slots[1] = -1                                                   # rotated, but kept out of the cache
    pos = rng.integers(0, 4096, T).astype(np.int32)
    pos[3] = -1                                                     # padding: not written anywhere
    ck = torch.full(h.kv_cache_shape(nb, bs), 3.0, dtype=torch.bfloat16, device="cuda")
    cv = ck.clone()
    out, ws = h.qk_norm_rope(qkv, torch.from_numpy(pos).cuda(), r, slot_mapping=torch.from_numpy(slots).cuda(),
                             cache_k=ck, cache_v=cv)
    # the separate write of the rotated rows
    wk, wv = torch.full_like(ck, 3.0), torch.full_like(cv, 3.0)
    s2 = slots.copy()
    s2[3] = -1
    h.kv_cache_write(out, torch.from_numpy(s2).cuda(), wk, wv)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32)) == 0
    assert torch.equal(ck, wk) and torch.equal(cv, wv)


def test_replicated_kv_heads_and_full_width():
    # t = 8 over 2 kv heads: every shard rotates its own replica alike
    nq, nkv, t, T = 8, 2, 8, 6
    h = handle(nq, nkv, 128, t)
    r = tl.Rope(64, 128)
    qkv = workloads.draw((t, T, width(nq, nkv, 128, t)), 1, 0)
    pos = np.arange(T) * 9
    out, _ = h.qk_norm_rope(qkv.cuda(), torch.from_numpy(pos.astype(np.int32)).cuda(), r)
    check(out, qkv, pos, nq, nkv, 128, t, 128, dict(base=10000.0), False, None, None, 1e-6)


def test_values_at_the_ends():
    # zero heads stay zero under the norm, infinities and NaN stay in their own head
    h = handle(4, 2, 128, 1)
    r = tl.Rope(64, 128, q_gamma=gamma(128, 0).cuda(), k_gamma=gamma(128, 1).cuda(), eps=1e-6)
    qkv = workloads.draw((1, 2, 8 * 128), 5, 0).cuda()
    qkv[0, 0, 0:128] = 0
    qkv[0, 0, 128] = float("inf")
    qkv[0, 0, 256] = float("nan")
    out, _ = h.qk_norm_rope(qkv, torch.tensor([3, 5], dtype=torch.int32, device="cuda"), r)
    o = out[0].float().cpu().view(2, 8, 128)
    assert (o[0, 0] == 0).all() and torch.isnan(o[0, 1]).any() and torch.isnan(o[0, 2]).any()
    assert torch.isfinite(o[0, 3:]).all() and torch.isfinite(o[1]).all()


def test_bad_positions_and_slots_raise_the_status():
    h = handle(4, 2, 128, 1)
    r = tl.Rope(64, 128)
    qkv = workloads.draw((1, 3, 8 * 128), 5, 0).cuda()
    keep = torch.full_like(qkv, 9.0)
    _, ws = h.qk_norm_rope(qkv, torch.tensor([1, 64, 2], dtype=torch.int32, device="cuda"), r, out=keep)
    assert int(ws[:4].view(torch.int32)) == tl.TP_ERR_SHAPE
    assert (keep[:, 1] == 9.0).all() and not (keep[:, [0, 2]] == 9.0).all(-1).any()
    ck = torch.zeros(h.kv_cache_shape(2, 16), dtype=torch.bfloat16, device="cuda")
    cv = torch.zeros_like(ck)
    _, ws = h.qk_norm_rope(qkv, torch.tensor([1, 3, 2], dtype=torch.int32, device="cuda"), r,
                           slot_mapping=torch.tensor([31, 32, 0], dtype=torch.int32, device="cuda"), cache_k=ck, cache_v=cv)
    assert int(ws[:4].view(torch.int32)) == tl.TP_ERR_SHAPE
    full = ck.view(-1, 2, 128).abs().amax((1, 2)) > 0
    assert full.nonzero().flatten().tolist() == [0, 31]


def test_refusals():
    h, mlp_cfg = handle(4, 2, 128, 1), tl.make_config(tl.TP_BLOCK_MLP, 1, 64, 64)
    w = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    mlp = tl.TPLinear(mlp_cfg, [w, w, w])
    r = tl.Rope(64, 128)
    qkv = torch.zeros(1, 4, 8 * 128, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    L = tl.lib()

    def call(hd=h.handle, T=4, q=qkv.data_ptr(), o=qkv.data_ptr(), p=pos.data_ptr(), rope=r.args, slots=None, ck=None,
             cv=None, nb=0, bs=0, w=ws.data_ptr(), wb=16):
        return L.tp_qk_norm_rope(hd, T, q, o, p, None if rope is None else ctypes.byref(rope), slots, ck, cv, nb, bs, w, wb,
                                 None)

    def args(**kw):
        a = tl.RopeArgs(r.args.table, 64, 128, 0, None, None, 1e-6)
        for k, v in kw.items():
            setattr(a, k, v)
        return a
    assert call() == tl.TP_OK and call(T=0, q=None) == tl.TP_OK
    assert call(hd=mlp.handle) == tl.TP_ERR_ARG and call(T=-1) == tl.TP_ERR_SHAPE
    assert call(q=None) == tl.TP_ERR_ARG and call(o=qkv.data_ptr() + 8) == tl.TP_ERR_ARG
    assert call(o=qkv.data_ptr() + 1024) == tl.TP_ERR_ARG                       # overlaps
    assert call(p=None) == tl.TP_ERR_ARG and call(rope=None) == tl.TP_ERR_ARG and call(wb=8) == tl.TP_ERR_ARG
    assert call(rope=args(table=None)) == tl.TP_ERR_ARG and call(rope=args(n_pos=0)) == tl.TP_ERR_SHAPE
    for rd in (0, 3, 130, -2):
        assert call(rope=args(rotary_dim=rd)) == tl.TP_ERR_SHAPE
    assert call(rope=args(layout=2)) == tl.TP_ERR_ARG and call(rope=args(eps=-1.0)) == tl.TP_ERR_ARG
    assert call(rope=args(q_gamma=r.args.table + 2)) == tl.TP_ERR_ARG
    assert call(slots=pos.data_ptr()) == tl.TP_ERR_SHAPE                        # no blocks
    assert call(slots=pos.data_ptr(), nb=1, bs=16) == tl.TP_ERR_ARG             # no caches
    assert call(slots=pos.data_ptr() + 2, nb=1, bs=16, ck=qkv.data_ptr(), cv=qkv.data_ptr()) == tl.TP_ERR_ARG
    assert call(slots=pos.data_ptr(), nb=1 << 31, bs=16, ck=qkv.data_ptr(), cv=qkv.data_ptr()) == tl.TP_ERR_UNSUPPORTED
    h64 = handle(4, 2, 64, 1)
    assert call(hd=h64.handle, rope=args(rotary_dim=64), slots=pos.data_ptr(), nb=1, bs=16, ck=qkv.data_ptr(),
                cv=qkv.data_ptr()) == tl.TP_ERR_UNSUPPORTED                     # the cache holds 128
    h264 = handle(2, 1, 264, 1)
    assert call(hd=h264.handle) == tl.TP_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        h.qk_norm_rope(qkv[..., :128], pos, r)
    with pytest.raises(TypeError):
        h.qk_norm_rope(qkv, pos.long(), r)
    with pytest.raises(ValueError):
        h.qk_norm_rope(qkv, pos[:3], r)
    with pytest.raises(ValueError):
        h.qk_norm_rope(qkv, pos, r, slot_mapping=pos)
    with pytest.raises(ValueError):
        tl.Rope(64, 128, scaling="spiral")
    with pytest.raises(ValueError):
        tl.Rope(64, 128, q_gamma=gamma(128, 0).cuda(), k_gamma=gamma(64, 0).cuda())
    with pytest.raises(ValueError):                                             # weights of other heads
        h.qk_norm_rope(qkv, pos, tl.Rope(64, 64, k_gamma=gamma(64, 0).cuda()))
    with pytest.raises(ValueError):
        h.qk_norm_rope(qkv, pos, r, out=torch.zeros(1, 4, 7 * 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        mlp.qk_norm_rope(qkv, pos, r)
    torch.cuda.synchronize()
