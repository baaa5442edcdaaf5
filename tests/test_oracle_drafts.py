"""Pins of the rotary, token-tree and page-move oracles, and the host side of those calls (CPU only).

Rotation: it keeps every pair's length, q . k depends on the positions' difference alone,
position 0 changes nothing, and the rotation by p then by p' is the one by p + p'. The
library's frequencies (host code) equal the oracle's. Tree attention: a chain is the causal
paged attention; a tree's branches are the chains of its paths; NaN in places a token does
not see has no effect. Host refusals of every call need no GPU.
"""
import ctypes
import math

import numpy as np
import pytest

import oracle
import tensor_linear_layers_gb300 as tl
from oracle import drafts, rope
from tests.test_oracle_kv_cache import _setup

SCALINGS = [
    dict(scaling="none"), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
    dict(scaling="bands", factor=8.0, original=8192), dict(scaling="yarn", factor=16.0, original=4096),
    dict(scaling="yarn", factor=0.5, original=4096), dict(scaling="bands", factor=2.0, original=1, low=0.5, high=0.75),
]


@pytest.fixture(scope="module")
def L():
    from tensor_linear_layers_gb300 import _build
    _build.build()
    return tl.lib()


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("d,base", [(128, 500000.0), (64, 10000.0), (20, 10000.0), (4, 1.5), (256, 1e6)])
def test_library_frequencies_equal_the_oracles(L, kw, d, base):
    f, m = oracle.rope_frequencies(d, base, **kw)
    cfg = tl.RopeConfig(d, tl.ROPE_SCALINGS[kw["scaling"]], base, kw.get("factor", 1.0), kw.get("low", 1.0),
                        kw.get("high", 4.0), 1.0, 32.0, 0.0, kw.get("original", 0))
    got, gm = tl.rope_frequencies(cfg)
    np.testing.assert_allclose(got, f, rtol=1e-13)
    assert gm == pytest.approx(m, rel=1e-15)
    cfg.attn_factor = 1.25
    assert tl.rope_frequencies(cfg)[1] == 1.25


@pytest.mark.parametrize("change,code", [
    (dict(rotary_dim=3), tl.TP_ERR_SHAPE), (dict(rotary_dim=0), tl.TP_ERR_SHAPE), (dict(rotary_dim=258), tl.TP_ERR_SHAPE),
    (dict(scaling=5), tl.TP_ERR_ARG), (dict(scaling=-1), tl.TP_ERR_ARG), (dict(base=1.0), tl.TP_ERR_ARG),
    (dict(base=math.nan), tl.TP_ERR_ARG), (dict(base=math.inf), tl.TP_ERR_ARG),
    (dict(scaling=1, factor=0.0), tl.TP_ERR_ARG), (dict(scaling=4, factor=math.nan), tl.TP_ERR_ARG),
    (dict(scaling=2, rotary_dim=2), tl.TP_ERR_SHAPE), (dict(scaling=3, original_max_position=0), tl.TP_ERR_ARG),
    (dict(scaling=3, low_freq_factor=4.0), tl.TP_ERR_ARG), (dict(scaling=4, beta_slow=0.0), tl.TP_ERR_ARG),
    (dict(scaling=4, beta_fast=1.0), tl.TP_ERR_ARG), (dict(attn_factor=-1.0), tl.TP_ERR_ARG),
])
def test_bad_rope_configurations_are_refused(L, change, code):
    cfg = tl.RopeConfig(128, 0, 10000.0, 8.0, 1.0, 4.0, 1.0, 32.0, 0.0, 4096)
    tl.rope_frequencies(cfg)
    for k, v in change.items():
        setattr(cfg, k, v)
    with pytest.raises(tl.TPError) as e:
        tl.rope_frequencies(cfg)
    assert e.value.code == code
    # the table refuses the same before it touches the device
    assert L.tp_rope_table(ctypes.byref(cfg), 16, ctypes.c_void_p(0x10000), None) == code


def test_rope_table_refuses_sizes_and_pointers(L):
    cfg = tl.RopeConfig(128, 0, 10000.0)
    p = ctypes.c_void_p(0x10000)
    assert L.tp_rope_table(None, 16, p, None) == tl.TP_ERR_ARG
    assert L.tp_rope_table(ctypes.byref(cfg), 0, p, None) == tl.TP_ERR_SHAPE
    assert L.tp_rope_table(ctypes.byref(cfg), 1 << 31, p, None) == tl.TP_ERR_SHAPE
    assert L.tp_rope_table(ctypes.byref(cfg), 16, None, None) == tl.TP_ERR_ARG
    assert L.tp_rope_table(ctypes.byref(cfg), 16, ctypes.c_void_p(0x10004), None) == tl.TP_ERR_ARG


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_depends_on_differences(interleaved):
    rng = np.random.default_rng(0)
    f, _ = oracle.rope_frequencies(12, 10000.0)
    q, k = rng.standard_normal((1, 16)), rng.standard_normal((1, 16))

    def at(x, p):
        return rope.rotate_pairs(x, np.array([[float(p)]]) * f, interleaved)
    np.testing.assert_allclose(at(q, 0), q, rtol=0)
    np.testing.assert_allclose(np.linalg.norm(at(q, 77)), np.linalg.norm(q), rtol=1e-14)
    np.testing.assert_allclose(at(at(q, 5), 30), at(q, 35), atol=1e-13)
    assert (at(q, 9)[0, 12:] == q[0, 12:]).all()
    d = at(q, 1000) @ at(k, 993).T
    np.testing.assert_allclose(at(q, 107) @ at(k, 100).T, d, atol=1e-12)
    assert abs((at(q, 108) @ at(k, 100).T - d).item()) > 1e-4      # a position off by one is seen


def test_layouts_are_permutations_of_each_other():
    rng = np.random.default_rng(1)
    f, m = oracle.rope_frequencies(8, 10000.0, "yarn", 4.0, 64)
    x, ang = rng.standard_normal((3, 8)), np.array([[1.0], [5.0], [9.0]]) * f
    perm = np.array([0, 2, 4, 6, 1, 3, 5, 7])                       # interleaved -> half
    a = rope.rotate_pairs(x, ang, True, m)[:, perm]
    np.testing.assert_allclose(a, rope.rotate_pairs(x[:, perm], ang, False, m), rtol=1e-14)


def test_qk_norm_rope_touches_q_and_k_heads_alone():
    rng = np.random.default_rng(2)
    nq, nkv, hd, t, T = 4, 2, 8, 2, 3
    a = rng.standard_normal((t, T, 4 * hd))
    f, _ = oracle.rope_frequencies(6, 100.0)
    g = np.linspace(0.5, 1.5, hd)
    out = oracle.qk_norm_rope(a, [0, -1, 7], f, nq, nkv, hd, t, k_gamma=g, eps=1e-3)
    np.testing.assert_array_equal(out[:, :, 3 * hd:], a[:, :, 3 * hd:])         # v
    np.testing.assert_array_equal(out[:, 1], a[:, 1])                           # padding token
    np.testing.assert_allclose(out[:, 0, :2 * hd], a[:, 0, :2 * hd])            # q at position 0, no gamma
    k = a[1, 2, 2 * hd:3 * hd]
    want = rope.rotate_pairs((k / np.sqrt((k * k).mean() + 1e-3) * g)[None], 7.0 * f[None], False)[0]
    np.testing.assert_allclose(out[1, 2, 2 * hd:3 * hd], want)


def test_a_chain_is_causal_paged_attention():
    nq, nkv, hd, t, lens, new, bs = 4, 2, 4, 2, [5, 9, 1], [2, 4, 1], 4
    _, tables, ck, cv, qkv, qsl = _setup(nq, nkv, hd, t, lens, new, bs, 3)
    sees = [oracle.tree_sees(list(range(-1, n - 1))) for n in new]
    got = oracle.tree_attention(qkv, qsl, lens, tables, sees, ck, cv, nq, nkv, hd, t, bs)
    want = oracle.paged_attention(qkv, qsl, lens, tables, ck, cv, nq, nkv, hd, t, bs)
    np.testing.assert_allclose(got, want, rtol=1e-12, atol=1e-12)


def test_a_branch_is_the_chain_of_its_path_and_the_rest_has_no_effect():
    nq, nkv, hd, t, bs = 4, 2, 4, 1, 2
    parents = [-1, 0, 0, 1, 2, -1]
    _, tables, ck, cv, qkv, _ = _setup(nq, nkv, hd, t, [7 + 6], [6], bs, 4)
    sees = oracle.tree_sees(parents)
    np.testing.assert_array_equal(np.nonzero(sees[4])[0], [0, 2, 4])
    got = oracle.tree_attention(qkv, [0, 6], [13], tables, [sees], ck, cv, nq, nkv, hd, t, bs)
    # the same path 0, 2, 4 as a chain of three after the 7 cached tokens
    path, row = [0, 2, 4], list(tables[0])
    k2, v2 = ck.copy(), cv.copy()
    for j, i in enumerate(path):
        s, d = oracle.slot_of([row], 0, 7 + i, bs), oracle.slot_of([row], 0, 7 + j, bs)
        k2[:, d // bs, d % bs], v2[:, d // bs, d % bs] = ck[:, s // bs, s % bs], cv[:, s // bs, s % bs]
    want = oracle.paged_attention(qkv[:, path], [0, 3], [10], tables, k2, v2, nq, nkv, hd, t, bs)
    np.testing.assert_allclose(got[:, path], want, rtol=1e-12, atol=1e-12)
    s = oracle.slot_of(tables, 0, 7 + 3, bs)                        # token 3 is on another branch
    cv[:, s // bs, s % bs] = np.nan
    again = oracle.tree_attention(qkv, [0, 6], [13], tables, [sees], ck, cv, nq, nkv, hd, t, bs)
    assert np.isfinite(again[:, [0, 1, 2, 4, 5]]).all() and np.isnan(again[:, 3]).all()


def test_mask_words_and_empty_rows():
    sees = oracle.tree_sees([-1] + list(range(39)))                 # a chain of 40
    w = oracle.mask_words(sees, 2)
    assert w.dtype == np.int32 and w[31, 0] == -1 and w[31, 1] == 0 and w[39, 1] == 255
    with pytest.raises(ValueError):
        oracle.tree_sees([0])
    _, tables, ck, cv, qkv, qsl = _setup(2, 1, 4, 1, [2], [2], 4, 5)
    out = oracle.tree_attention(qkv, qsl, [2], tables, [np.array([[False, False], [True, False]])], ck, cv, 2, 1, 4, 1, 4)
    assert (out[:, 0] == 0).all() and (out[:, 1] != 0).any()


def test_compact_in_place_equals_compact_to_a_copy():
    rng = np.random.default_rng(6)
    cache = rng.standard_normal((2, 9, 4, 1, 3))
    tables = np.array([[4, 1, 7, 0], [2, 8, 3, 6]])
    ctx, acc = [3, 6], [[0, 2, 3, 7], [5]]
    out = oracle.compact(cache, ctx, acc, tables, tables, 4)
    for b in range(2):
        flat_in = cache[:, tables[b]].reshape(2, -1, 3)
        flat_out = out[:, tables[b]].reshape(2, -1, 3)
        np.testing.assert_array_equal(flat_out[:, :ctx[b]], flat_in[:, :ctx[b]])
        for j, i in enumerate(acc[b]):
            np.testing.assert_array_equal(flat_out[:, ctx[b] + j], flat_in[:, ctx[b] + i])
    assert (oracle.copy_blocks(cache, [(-1, 3), (2, 5)])[:, 5] == cache[:, 2]).all()


def test_calls_refuse_a_null_handle(L):
    p, n = ctypes.c_void_p(0x10000), ctypes.c_int64()
    arr = (ctypes.c_void_p * 1)(0x10000)
    r = tl.RopeArgs(0x10000, 16, 128, 0, None, None, 1e-6)
    assert L.tp_qk_norm_rope(None, 4, p, p, p, ctypes.byref(r), None, None, None, 0, 0, p, 16, None) == tl.TP_ERR_ARG
    assert L.tp_layer_set_rope(None, ctypes.byref(r), p) == tl.TP_ERR_ARG
    assert L.tp_tree_attention_workspace_size(None, 1, 8, 64, ctypes.byref(n)) == tl.TP_ERR_ARG
    assert L.tp_tree_attention(None, 4, p, p, p, 1, 4, 64, p, 4, p, 1, p, p, 8, 16, p, p, 1 << 20, None) == tl.TP_ERR_ARG
    assert L.tp_kv_cache_copy_blocks(None, p, 1, 1, arr, arr, 8, 16, p, 16, None) == tl.TP_ERR_ARG
    assert L.tp_kv_cache_compact(None, 1, p, p, p, 4, p, p, 4, 1, arr, arr, 8, 16, p, p, 16, None) == tl.TP_ERR_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), tl.TP_ERR_SHAPE), (dict(n_reqs=0), tl.TP_ERR_SHAPE), (dict(mq=0), tl.TP_ERR_SHAPE),
    (dict(mq=257, words=9), tl.TP_ERR_UNSUPPORTED), (dict(mq=33), tl.TP_ERR_SHAPE), (dict(words=0), tl.TP_ERR_SHAPE),
    (dict(parents=None), tl.TP_ERR_ARG), (dict(mask=0x10002), tl.TP_ERR_ARG), (dict(pos=0x10001), tl.TP_ERR_ARG),
    (dict(ws_bytes=8), tl.TP_ERR_ARG), (dict(ws=0x10004), tl.TP_ERR_ARG),
])
def test_tree_mask_refuses(L, kw, code):
    a = dict(T=4, n_reqs=1, mq=4, parents=0x10000, words=1, mask=0x10000, pos=None, ws=0x10000, ws_bytes=16)
    a.update(kw)

    def v(x):
        return None if x is None else ctypes.c_void_p(x)
    rc = L.tp_tree_mask(a["T"], a["n_reqs"], a["mq"], v(a["parents"]), v(0x10000), v(0x10000), v(a["mask"]), a["words"],
                        v(a["pos"]), v(a["ws"]), a["ws_bytes"], None)
    assert rc == code


def test_tree_mask_of_no_tokens_enqueues_nothing(L):
    assert L.tp_tree_mask(0, 0, 0, None, None, None, None, 0, None, None, 0, None) == tl.TP_OK
