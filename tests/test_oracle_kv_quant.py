"""Pins of the oracle of the 8-bit cache and of attention with a window (oracle/kv_quant.py)."""
import numpy as np
import pytest
import torch

import oracle
from oracle.kv_quant import E_HI, E_LO, sees


def test_e4m3_values_are_the_formats():
    # torch's own conversion of every code, and the landmarks of the format
    bits = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double().numpy()
    np.testing.assert_array_equal(oracle.e4m3_values(), bits)
    v = oracle.e4m3_values()
    assert v[0x7e] == 448 and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6 and v[0x38] == 1.0


def test_rounding_is_to_nearest_even():
    v = oracle.e4m3_values()[:127]
    np.testing.assert_array_equal(oracle.round_e4m3(v), v)
    mid = (v[:-1] + v[1:]) / 2
    want = np.where(np.arange(126) % 2 == 0, v[:-1], v[1:])
    np.testing.assert_array_equal(oracle.round_e4m3(mid), want)
    np.testing.assert_array_equal(oracle.round_e4m3(-mid), -want)
    x = np.random.default_rng(0).standard_normal(4000) * np.exp(np.random.default_rng(1).uniform(-6, 6, 4000))
    got = torch.from_numpy(x.astype(np.float32)).clamp(-448, 448).to(torch.float8_e4m3fn).float().double().numpy()
    np.testing.assert_array_equal(oracle.round_e4m3(x.astype(np.float32)), got)
    assert oracle.round_e4m3(np.array([1e9, -465.0])).tolist() == [448, -448]


def test_scales_are_the_smallest_powers_that_hold_the_row():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((300, 128)) * np.exp2(rng.integers(-130, 120, 300))[:, None]
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    x[0] = 0
    x[1], x[2] = 448.0, 450.0
    y, s = oracle.quantise(x)
    e, top = s - 127, np.abs(x).max(-1)
    held = top <= 448 * np.exp2(e.astype(float))
    assert held[e < E_HI].all() and (s >= E_LO + 127).all()
    assert (top > 448 * np.exp2(e - 1.0))[e > E_LO].all()
    assert s[0] == 27 and s[1] == 127 and s[2] == 128
    # half a step of a code's value: 2^-4 of it, or of the smallest normal value
    back = oracle.values(y, s)
    assert (np.abs(back - x) <= 2.0 ** -4 * np.maximum(np.abs(x), np.exp2(e - 6.0)[:, None]))[e < E_HI].all()
    # a value is a bf16
    inside = (e > -100) & (e < 118)
    np.testing.assert_array_equal(torch.from_numpy(back[inside]).to(torch.bfloat16).double().numpy(), back[inside])


def test_rows_that_are_not_finite():
    x = np.ones((3, 128))
    x[0, 5], x[1, 7] = np.nan, -np.inf
    y, s = oracle.quantise(x)
    assert s.tolist() == [255, 255, 119] and (y[:2] == 0).all()
    v = oracle.values(y, s)
    assert np.isnan(v[:2]).all() and (v[2] == 1).all()


def test_sees_by_hand():
    assert sees(5, 8, 0, 0).tolist() == [True] * 6 + [False] * 2
    assert sees(5, 8, 2, 0).nonzero()[0].tolist() == [4, 5]
    assert sees(5, 8, 2, 1).nonzero()[0].tolist() == [0, 4, 5]
    assert sees(5, 8, 1, 9).nonzero()[0].tolist() == [0, 1, 2, 3, 4, 5]
    assert sees(0, 8, 1, 0).nonzero()[0].tolist() == [0]


def case(nq, nkv, t, n, ctx, bs, seed):
    rng = np.random.default_rng(seed)
    q_per, kv_per, _ = oracle.gqa_partition(nq, nkv, t)
    lens = [c + k for c, k in zip(ctx, n)]
    blocks = sum(-(-x // bs) for x in lens) + 2
    perm, at, tables = rng.permutation(blocks), 0, np.zeros((len(n), max(-(-x // bs) for x in lens)), dtype=int)
    for b, x in enumerate(lens):
        k = -(-x // bs)
        tables[b, :k] = perm[at:at + k]
        at += k
    qsl = np.concatenate([[0], np.cumsum(n)])
    qkv = rng.standard_normal((t, qsl[-1], (q_per + 2 * kv_per) * 8))
    ck, cv = (rng.standard_normal((t, blocks, bs, kv_per, 8)) for _ in range(2))
    return qkv, qsl, lens, tables, ck, cv


@pytest.mark.parametrize("nq,nkv,t", [(4, 2, 2), (4, 1, 2), (6, 2, 1)])
def test_without_a_window_it_is_the_paged_attention(nq, nkv, t):
    c = case(nq, nkv, t, [1, 5, 0, 3], [7, 0, 4, 12], 4, 3)
    np.testing.assert_allclose(oracle.chunk_attention(*c, nq, nkv, 8, t, 4), oracle.paged_attention(*c, nq, nkv, 8, t, 4),
                               atol=1e-12)
    np.testing.assert_allclose(oracle.chunk_attention(*c, nq, nkv, 8, t, 4, window=99), oracle.paged_attention(*c, nq, nkv, 8, t, 4),
                               atol=1e-12)


def test_a_window_is_attention_over_what_is_left():
    # element by element, with loops
    nq, nkv, t, bs, W, S = 4, 2, 2, 4, 3, 2
    qkv, qsl, lens, tables, ck, cv = case(nq, nkv, t, [2, 6], [9, 0], bs, 4)
    got = oracle.chunk_attention(qkv, qsl, lens, tables, ck, cv, nq, nkv, 8, t, bs, W, S)
    for b in range(2):
        for i in range(qsl[b], qsl[b + 1]):
            p = lens[b] - (qsl[b + 1] - i)
            for r in range(t):
                for h in range(2):
                    num, den = np.zeros(8), 0.0
                    for j in range(lens[b]):
                        if j > p or (j <= p - W and j >= S):
                            continue
                        blk, off = tables[b, j // bs], j % bs
                        e = np.exp(sum(qkv[r, i, h * 8 + d] * ck[r, blk, off, 0, d] for d in range(8)) / np.sqrt(8))
                        num, den = num + e * cv[r, blk, off, 0], den + e
                    np.testing.assert_allclose(got[r, i, h * 8:h * 8 + 8], num / den, atol=1e-12)


def test_a_window_of_one_returns_the_tokens_own_value():
    qkv, qsl, lens, tables, ck, cv = case(2, 1, 1, [3], [5], 4, 5)
    got = oracle.chunk_attention(qkv, qsl, lens, tables, ck, cv, 2, 1, 8, 1, 4, window=1)
    for i in range(3):
        p = 5 + i
        np.testing.assert_allclose(got[0, i, :8], cv[0, tables[0, p // 4], p % 4, 0], atol=1e-12)


@pytest.mark.parametrize("wrong", [dict(window=4, sinks=2), dict(window=3, sinks=1), dict(window=2, sinks=2)])
def test_planted_mistakes_are_caught(wrong):
    c = case(4, 2, 2, [2, 6], [9, 0], 4, 4)
    a = oracle.chunk_attention(*c, 4, 2, 8, 2, 4, window=3, sinks=2)
    assert np.abs(a - oracle.chunk_attention(*c, 4, 2, 8, 2, 4, **wrong)).max() > 1e-3
