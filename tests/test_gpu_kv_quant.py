"""The paged KV cache in 8 bits (tp_kv_quant_write, tp_kv_quant_read): every code and scale is the oracle's, every
value read back is exact, and nothing else is written."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import tensor_linear_layers_gb300 as tl

pytestmark = pytest.mark.gpu


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


def rows(t, T, width, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, T, width // 128, 128, generator=g)
    return (x * torch.exp(spread * torch.randn(t, T, width // 128, 1, generator=g))).to(torch.bfloat16).view(t, T, width)


def dirty(h, nb, bs, seed):
    """A cache of random bytes: (codes_k, codes_v, scales_k, scales_v) on the GPU."""
    g = torch.Generator().manual_seed(seed)
    shape = h.kv_cache_shape(nb, bs)
    return [torch.randint(0, 256, s, generator=g, dtype=torch.uint8).cuda().view(d)
            for s, d in ((shape, torch.float8_e4m3fn),) * 2 + ((shape[:-1], torch.uint8),) * 2]


def plain(cache):
    return [x.view(torch.uint8).cpu().numpy() for x in cache]


def written(before, qkv, slots, nq, nkv, t):
    """The cache's bytes after the oracle's write."""
    q_per, kv_per, _ = oracle.gqa_partition(nq, nkv, t)
    mags = oracle.e4m3_values()[:127]
    out = [x.copy() for x in before]
    heads = oracle.bf16_to_f64(qkv).reshape(t, qkv.shape[1], -1, 128)
    for i, s in enumerate(slots):
        if s < 0:
            continue
        for which in range(2):
            at = q_per + which * kv_per
            y, sc = oracle.quantise(heads[:, i, at:at + kv_per])
            code = np.searchsorted(mags, np.abs(y)) + 128 * (np.signbit(y) & True)
            out[which].reshape(t, -1, kv_per, 128)[:, s] = code
            out[2 + which].reshape(t, -1, kv_per)[:, s] = sc
    return out


def same(got, want):
    """Equal bytes, but that codes 0x00 and 0x80 are both zero."""
    for k, (a, b) in enumerate(zip(got, want)):
        if k < 2:
            a, b = np.where(a == 128, 0, a), np.where(b == 128, 0, b)
        assert np.array_equal(a, b), f"array {k}: {np.argwhere(a != b)[:5]}"


@pytest.mark.parametrize("nq,nkv,t,T,nb,bs", [
    (8, 2, 2, 1, 3, 16), (8, 2, 2, 37, 9, 16), (4, 4, 1, 130, 200, 1), (8, 1, 1, 5, 2, 3), (8, 2, 8, 33, 4, 24),
    (28, 4, 4, 1021, 40, 64), (64, 8, 8, 64, 3, 130),
    (32, 8, 1, 2600, 166, 16),             # more than eight rows per lane group and SM: four rows each, a last block half full
])
@pytest.mark.parametrize("gathered", [False, True])
def test_write_is_the_oracles_bit_for_bit(nq, nkv, t, T, nb, bs, gathered):
    h = handle(nq, nkv, t, tl.TP_FLAG_GATHERED if gathered else 0)
    q_per, kv_per, _ = oracle.gqa_partition(nq, nkv, t)
    qkv = rows(t, T, (q_per + 2 * kv_per) * 128, seed=T, spread=3.0)
    rng = np.random.default_rng(T)
    slots = rng.permutation(nb * bs)[:T].astype(np.int64)
    slots = np.concatenate([slots, -np.ones(max(0, T - len(slots)), dtype=np.int64)])
    slots[rng.random(T) < 0.1] = -1                          # padding tokens
    cache = dirty(h, nb, bs, T)
    want = written(plain(cache), qkv, slots, nq, nkv, t)
    x = qkv.permute(1, 0, 2).reshape(T, -1).contiguous() if gathered else qkv
    ws = h.kv_quant_write(x.cuda(), dev(slots), *cache)
    assert status(ws) == 0
    got = plain(cache)
    # slots not written keep every bit
    mask = np.ones(nb * bs, dtype=bool)
    mask[slots[slots >= 0]] = False
    for a, b in zip(got, want):
        assert np.array_equal(a.reshape(t, nb * bs, -1)[:, mask], b.reshape(t, nb * bs, -1)[:, mask])
    same(got, want)


def test_write_of_borders_ties_and_values_that_are_not_finite():
    nq, nkv, t = 2, 1, 1
    h = handle(nq, nkv, t)
    b = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    finite = b[torch.isfinite(b.float())]
    T = 700
    x = torch.zeros(T, 4, 128, dtype=torch.bfloat16)
    rng = np.random.default_rng(0)
    for i in range(400):                                    # every size of rows, ties among them (bf16 halves of steps)
        pick = finite[torch.from_numpy(rng.integers(0, len(finite), 256))]
        top = float(np.exp2(rng.integers(-133, 128)))
        x[i, 2:] = torch.where(pick.float().abs() <= top, pick, torch.zeros_like(pick)).view(2, 128)
    steps = torch.tensor([c + 0.5 * d for c, d in ((448, 0), (448, 4), (240, 32), (15, 2), (1.0625, 0), (2.0 ** -9, 0),
                                                    (2.0 ** -10, 0), (1.5 * 2.0 ** -9, 0), (2.5 * 2.0 ** -9, 0))])
    for i in range(400, 600):
        x[i, 2:, :9] = (steps * 2.0 ** int(rng.integers(-90, 100))).to(torch.bfloat16)
        x[i, 2:, 9:] = -x[i, 2:, 0:1]
    x[600:, 2:] = 1.0
    for i, v in enumerate((float("nan"), float("inf"), -float("inf"), 3.38e38, -3.38e38, 1e-40, 0.0, 9.2e-41)):
        x[600 + i, 2, i * 16 + 3] = v
        x[620 + i, 3, :] = v
    qkv = x.view(1, T, 512)
    cache = dirty(h, 50, 16, 1)
    slots = np.arange(T)[::-1].copy()
    want = written(plain(cache), qkv, slots, nq, nkv, t)
    ws = h.kv_quant_write(qkv.cuda(), dev(slots), *cache)
    assert status(ws) == 0
    same(plain(cache), want)
    s = plain(cache)[2].reshape(-1)
    assert [int(s[slots[600 + i]]) for i in range(3)] == [255] * 3 and int(s[slots[606]]) == 119


@pytest.mark.parametrize("nq,nkv,t,n,nb,bs", [
    (8, 2, 2, 1, 3, 16), (4, 4, 1, 130, 7, 1), (8, 2, 8, 33, 4, 24), (28, 4, 4, 1021, 40, 64), (32, 8, 1, 2600, 10, 130)])
def test_read_is_exact(nq, nkv, t, n, nb, bs):
    h = handle(nq, nkv, t)
    kv_per = oracle.gqa_partition(nq, nkv, t)[1]
    rng = np.random.default_rng(n)
    cache = dirty(h, nb, bs, n)
    for c in cache[:2]:
        u = c.view(torch.uint8)
        u[(u & 127) == 127] = 5                              # no NaN codes: the write makes none
    scales = [torch.from_numpy(rng.integers(10, 246, s.shape).astype(np.uint8)).cuda() for s in cache[2:]]
    scales[0][:, 0], scales[1][:, -1] = 0, 255
    cache = cache[:2] + scales
    slots = rng.integers(0, nb * bs, n)                      # repeated among them
    slots[rng.random(n) < 0.1] = -1
    slots[0] = 0
    k, v, ws = h.kv_quant_read(dev(slots), *cache)
    assert status(ws) == 0
    codes = oracle.e4m3_values()
    for got, c, s in ((k, cache[0], cache[2]), (v, cache[1], cache[3])):
        c, s = c.view(torch.uint8).cpu().numpy().reshape(t, -1, kv_per, 128), s.cpu().numpy().reshape(t, -1, kv_per)
        want = oracle.values(codes[c[:, slots]], s[:, slots])
        want[:, slots < 0] = 0
        # (values under 2^-126 are rounded to bf16 as subnormal numbers: scale byte 0 with small codes)
        want = torch.from_numpy(want).to(torch.float32).to(torch.bfloat16).float().numpy()
        np.testing.assert_array_equal(got.float().cpu().numpy(), want)


def test_read_returns_what_was_written():
    # through both calls a finite row comes back within half a step of its codes
    h = handle(8, 2, 2)
    qkv = rows(2, 300, 6 * 128, 7, 2.0)
    cache = h.kv_quant_cache(30, 16)
    slots = dev(np.random.default_rng(1).permutation(480)[:300])
    assert status(h.kv_quant_write(qkv.cuda(), slots, *cache)) == 0
    k, v, ws = h.kv_quant_read(slots, *cache)
    assert status(ws) == 0
    x = qkv.view(2, 300, 6, 128).float()
    for got, want in ((k, x[:, :, 4:5]), (v, x[:, :, 5:6])):
        top = want.abs().amax(-1, keepdim=True)
        # half a step is 2^-4 of a value, or under the smallest normal code half of 2^-9 * 2^e; top > 224 * 2^e, so
        # that half step of 2^-10 * 2^e is under top * 2^-10 / 224
        ok = (got.float().cpu() - want).abs() <= torch.maximum(want.abs() * 2.0 ** -4, top * (2.0 ** -10 / 224))
        assert bool(ok.all())


def test_slots_past_the_cache_and_no_tokens():
    h = handle(8, 2, 2)
    qkv = rows(2, 4, 6 * 128, 3).cuda()
    cache = dirty(h, 3, 16, 2)
    before = plain(cache)
    ws = h.kv_quant_write(qkv, dev([48, -1, 1 << 30, -5]), *cache)
    assert status(ws) == tl.TP_ERR_SHAPE
    for a, b in zip(plain(cache), before):
        assert np.array_equal(a, b)
    k, v, ws = h.kv_quant_read(dev([48, -1, 3]), *h.kv_quant_cache(3, 16))
    assert status(ws) == tl.TP_ERR_SHAPE and (k == 0).all() and (v == 0).all()
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    k, v, ws = h.kv_quant_read(e, *cache)
    assert status(ws) == 0 and k.shape == (2, 0, 1, 128)
    assert status(h.kv_quant_write(qkv[:, :0].contiguous(), e, *cache)) == 0


def test_captured_and_on_a_stream_of_its_own():
    h = handle(8, 2, 2)
    qkv, slots = rows(2, 20, 6 * 128, 9).cuda(), dev(np.arange(20))
    want = h.kv_quant_cache(2, 16)
    h.kv_quant_write(qkv, slots, *want)
    k0, v0, _ = h.kv_quant_read(slots, *want)
    cache, st, g = h.kv_quant_cache(2, 16), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        w1 = h.kv_quant_write(qkv, slots, *cache, stream=st)
        k, v, w2 = h.kv_quant_read(slots, *cache, stream=st)
    for _ in range(2):
        for x in (k, v, *(c.view(torch.uint8) for c in cache)):
            x.zero_()
        g.replay()
        assert status(w1) == 0 and status(w2) == 0
        assert torch.equal(k, k0) and torch.equal(v, v0)
        for a, b in zip(plain(cache), plain(want)):
            assert np.array_equal(a, b)


def test_refusals():
    h, h64, L = handle(8, 2, 2), handle(8, 2, 2, hd=64), tl.lib()

    def at(x):
        return None if x is None else ctypes.c_void_p(x)

    def write(hd=h.handle, T=8, q=1 << 24, slots=1 << 20, ck=1 << 25, cv=1 << 26, sk=1 << 27, sv=1 << 28, nb=8, bs=16,
              ws=1 << 16, wb=16):
        return L.tp_kv_quant_write(hd, T, at(q), at(slots), at(ck), at(cv), at(sk), at(sv), nb, bs, at(ws), wb, None)

    def read(hd=h.handle, T=8, slots=1 << 20, ck=1 << 25, cv=1 << 26, sk=1 << 27, sv=1 << 28, nb=8, bs=16, k=1 << 29,
             v=1 << 30, ws=1 << 16, wb=16):
        return L.tp_kv_quant_read(hd, T, at(slots), at(ck), at(cv), at(sk), at(sv), nb, bs, at(k), at(v), at(ws), wb, None)
    for f, outs in ((write, ("q",)), (read, ("k", "v"))):
        assert f(T=0) == tl.TP_OK and f(T=-1) == tl.TP_ERR_SHAPE and f(T=(1 << 24) + 1) == tl.TP_ERR_UNSUPPORTED
        assert f(hd=None) == tl.TP_ERR_ARG and f(hd=h64.handle) == tl.TP_ERR_UNSUPPORTED
        assert f(nb=0) == tl.TP_ERR_SHAPE and f(bs=0) == tl.TP_ERR_SHAPE and f(nb=1 << 31) == tl.TP_ERR_UNSUPPORTED
        assert f(nb=1 << 27) == tl.TP_ERR_UNSUPPORTED and f(wb=8) == tl.TP_ERR_ARG and f(ws=None) == tl.TP_ERR_ARG
        for k in ("ck", "cv") + outs:
            assert f(**{k: None}) == tl.TP_ERR_ARG and f(**{k: (1 << 25) + 8}) == tl.TP_ERR_ARG
        assert f(sk=None) == tl.TP_ERR_ARG and f(sv=None) == tl.TP_ERR_ARG
        assert f(slots=None) == tl.TP_ERR_ARG and f(slots=(1 << 20) + 2) == tl.TP_ERR_ARG
    for bad in (dict(ck=1 << 24), dict(cv=1 << 25), dict(sk=(1 << 25) + 5), dict(sv=1 << 27), dict(cv=1 << 20)):
        assert write(**bad) == tl.TP_ERR_ARG and b"overlaps" in L.tp_last_error()
    for bad in (dict(k=1 << 25), dict(v=1 << 29), dict(k=1 << 27), dict(v=1 << 20)):
        assert read(**bad) == tl.TP_ERR_ARG and b"overlaps" in L.tp_last_error()
    cache = h.kv_quant_cache(2, 16)
    qkv, slots = rows(2, 4, 6 * 128, 3).cuda(), dev(np.arange(4))
    with pytest.raises(TypeError):
        h.kv_quant_write(qkv, slots.long(), *cache)
    with pytest.raises(ValueError):
        h.kv_quant_write(qkv, slots[:3], *cache)
    with pytest.raises(ValueError):
        h.kv_quant_write(qkv, slots, cache[0].view(torch.uint8), *cache[1:])
    with pytest.raises(ValueError):
        h.kv_quant_write(qkv, slots, *cache[:3], cache[3][:, :1])
    with pytest.raises(ValueError):
        h.kv_quant_read(slots, *cache, out=(torch.empty(2, 3, 1, 128, dtype=torch.bfloat16, device="cuda"),) * 2)
