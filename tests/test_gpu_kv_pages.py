"""Pages moved inside the paged KV cache (tp_kv_cache_copy_blocks, tp_kv_cache_compact): copies, bit for bit."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import workloads
import tensor_linear_layers_gb300 as tl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from tensor_linear_layers_gb300 import _build
    _build.build()
    tl.lib()
    torch.cuda.set_device(0)


def handle(nq, nkv, t, hd=128, H=64):
    cfg = tl.make_config(tl.TP_BLOCK_ATTN_PROJ, t, H, n_q_heads=nq, n_kv_heads=nkv, head_dim=hd)
    z = torch.zeros(nq * hd, H, dtype=torch.bfloat16, device="cuda")
    return tl.TPLinear(cfg, [z, z[:nkv * hd].contiguous(), z[:nkv * hd].contiguous(), z.t().contiguous()])


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def status(ws):
    torch.cuda.synchronize()
    return int(ws[:4].view(torch.int32))


def caches(h, layers, nb, bs, seed):
    """Layers' caches with random bits (NaN patterns among them: copies keep them)."""
    g = torch.Generator().manual_seed(seed)
    shape = h.kv_cache_shape(nb, bs)
    one = [torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, dtype=torch.int16).view(torch.bfloat16)
           for _ in range(2 * layers)]
    return [x.cuda() for x in one[:layers]], [x.cuda() for x in one[layers:]]


def bits(x):
    return x.view(torch.int16).cpu().numpy()


@pytest.mark.parametrize("nq,nkv,t,layers,nb,bs,pairs", [
    (8, 2, 2, 1, 4, 16, [(0, 3)]),
    (8, 2, 4, 3, 9, 8, [(0, 3), (0, 4), (1, 8), (-1, 5), (-7, -1)]),       # a source twice, padding entries
    (4, 4, 1, 128, 5, 1, [(4, 0), (3, 1)]),                                # the most layers; blocks of one token
    (8, 4, 8, 2, 40, 24, [(i, 20 + i) for i in range(20)]),
    (8, 2, 1, 2, 6, 130, [(5, 0)]),                                        # large pages
    (8, 1, 1, 1, 3, 3, [(2, 2)]),                                          # a page onto itself
])
def test_copy_blocks(nq, nkv, t, layers, nb, bs, pairs):
    h = handle(nq, nkv, t)
    ck, cv = caches(h, layers, nb, bs, seed=nb)
    before = [bits(x) for x in ck + cv]
    ws = h.kv_cache_copy_blocks(dev(pairs), ck, cv)
    assert status(ws) == 0
    for a, b in zip(before, ck + cv):
        np.testing.assert_array_equal(bits(b), oracle.copy_blocks(a, pairs))


def test_copy_blocks_bad_ids_and_no_pairs():
    h = handle(8, 2, 2)
    ck, cv = caches(h, 2, 6, 16, seed=1)
    before = [bits(x) for x in ck + cv]
    assert status(h.kv_cache_copy_blocks(torch.zeros(0, 2, dtype=torch.int32, device="cuda"), ck, cv)) == 0
    pairs = [(6, 1), (0, 6), (0, -1), (2, 3)]
    assert status(h.kv_cache_copy_blocks(dev(pairs), ck, cv)) == tl.TP_ERR_SHAPE
    for a, b in zip(before, ck + cv):
        np.testing.assert_array_equal(bits(b), oracle.copy_blocks(a, [(2, 3)]))


def compact_case(h, ctx, n, accepted, bs, layers, seed, in_place, m=None):
    rng = np.random.default_rng(seed)
    lens = [c + k for c, k in zip(ctx, n)]
    cols = max(-(-max(lens) // bs), 1) + 1
    need = [-(-L // bs) for L in lens]
    nb = 2 * sum(need) + 2
    perm = rng.permutation(nb)
    src = np.full((len(ctx), cols), -3, dtype=np.int32)
    used = 0
    for b, k in enumerate(need):
        src[b, :k] = perm[used:used + k]
        used += k
    dst = src.copy()
    if not in_place:
        for b, k in enumerate(need):                   # the drafts' pages are not the request's own
            first = ctx[b] // bs
            dst[b, first:k] = perm[used:used + k - first]
            used += k - first
    ck, cv = caches(h, layers, nb, bs, seed)
    m = max(max((len(a) for a in accepted), default=1), 1) if m is None else m
    acc = np.full((len(ctx), m), -1, dtype=np.int32)
    for b, a in enumerate(accepted):
        acc[b, :len(a)] = a
    return dict(lens=lens, src=src, dst=dst, ck=ck, cv=cv, acc=acc, qsl=np.concatenate([[0], np.cumsum(n)]))


def run_compact(h, c, out=None):
    d_src = dev(c["src"])
    d_dst = d_src if c["src"] is c["dst"] else dev(c["dst"])
    return h.kv_cache_compact(dev(c["qsl"]), dev(c["lens"]), dev(c["acc"]), d_src, d_dst, c["ck"], c["cv"], out=out)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("nq,nkv,t,ctx,n,accepted,bs,layers,m", [
    (8, 2, 2, [5], [4], [[0, 2, 3]], 16, 1, None),
    (8, 2, 4, [0, 31, 100], [8, 3, 20], [[7], [], [0, 1, 2, 5, 19]], 8, 3, 20),        # no cached token; nothing kept
    (4, 4, 1, [17, 15], [64, 9], [list(range(1, 64)), [0, 1, 2, 3, 8]], 16, 2, None),  # a shift by one over pages
    (8, 4, 8, [3], [30], [list(range(0, 30, 3))], 1, 2, None),
    (8, 1, 1, [50], [256], [list(range(0, 256, 2))], 24, 1, 200),
    (8, 2, 1, [9, 10], [5, 0], [[0, 1, 2, 3, 4], []], 4, 128, None),                   # the whole path; no drafts
])
def test_compact(nq, nkv, t, ctx, n, accepted, bs, layers, m, in_place):
    h = handle(nq, nkv, t)
    c = compact_case(h, ctx, n, accepted, bs, layers, len(n) + bs, in_place, m)
    before = [bits(x) for x in c["ck"] + c["cv"]]
    new, ws = run_compact(h, c)
    assert status(ws) == 0
    assert new.tolist() == [x + len(a) for x, a in zip(ctx, accepted)]
    for a, b in zip(before, c["ck"] + c["cv"]):
        np.testing.assert_array_equal(bits(b), oracle.compact(a, ctx, accepted, c["src"], c["dst"], bs))


@pytest.mark.parametrize("in_place", [True, False])
def test_compact_of_more_blocks_than_one_wave(in_place):
    h, layers, bs = handle(8, 8, 8), 128, 8   # 128 strips of columns for each of 7 requests
    rng = np.random.default_rng(71)
    ctx, n = [0, 3, 8, 13, 29, 40, 1], [9, 12, 8, 20, 17, 0, 5]
    accepted = [sorted(rng.permutation(k)[:min(k, m)].tolist()) for k, m in zip(n, [4, 5, 8, 17, 0, 3, 1])]
    c = compact_case(h, ctx, n, accepted, bs, layers, 71, in_place, 20)
    before = [bits(x) for x in c["ck"] + c["cv"]]
    new, ws = run_compact(h, c)
    assert status(ws) == 0
    assert new.tolist() == [x + len(a) for x, a in zip(ctx, accepted)]
    for a, b in zip(before, c["ck"] + c["cv"]):
        np.testing.assert_array_equal(bits(b), oracle.compact(a, ctx, accepted, c["src"], c["dst"], bs))


def test_compact_bad_lists_end_there():
    h, bs, ctx = handle(8, 2, 2), 16, [5, 20, 7, 3, 2]
    good = [[0, 2], [1, 3], [0], [1], []]
    c = compact_case(h, ctx, [6, 6, 6, 6, 6], good, bs, 2, 9, True, m=4)
    c["acc"][0, 2] = 2                        # does not rise
    c["acc"][1, 2:4] = [6, 5]                 # past the drafts
    c["acc"][2, 1:3] = [5, 2]                 # falls
    kept = [[0, 2], [1, 3], [0, 5], [1], []]
    c["src"][3, 0] = c["src"][3, 0]
    before = [bits(x) for x in c["ck"] + c["cv"]]
    new, ws = run_compact(h, c)
    assert status(ws) == tl.TP_ERR_SHAPE
    assert new.tolist() == [x + len(a) for x, a in zip(ctx, kept)]
    for a, b in zip(before, c["ck"] + c["cv"]):
        np.testing.assert_array_equal(bits(b), oracle.compact(a, ctx, kept, c["src"], c["dst"], bs))


def test_compact_bad_pages_and_counts():
    h, bs = handle(8, 2, 2), 16
    c = compact_case(h, [5, 30, 40, 3], [6, 6, 6, 6], [[0, 2], [0, 1, 4], [0, 3], [2]], bs, 2, 9, False)
    c["src"][0, 0] = 10_000
    c["dst"][1, 2] = -1                       # positions 30, 31 are in block 1: two tokens are kept
    c["qsl"] = np.array([0, 6, 12, 18, 17])   # the last request has -1 drafts
    before = [bits(x) for x in c["ck"] + c["cv"]]
    new, ws = run_compact(h, c)
    assert status(ws) == tl.TP_ERR_SHAPE
    assert new.tolist() == [5, 32, 42, 9]
    kept = [[], [0, 1], [0, 3], []]
    for a, b in zip(before, c["ck"] + c["cv"]):
        np.testing.assert_array_equal(bits(b), oracle.compact(a, [5, 30, 40, 3], kept, c["src"], c["dst"], bs))
    d = compact_case(h, [5], [6], [[0]], bs, 1, 9, True)
    d["lens"] = [4]                           # fewer tokens than drafts
    new, ws = run_compact(h, d)
    assert status(ws) == tl.TP_ERR_SHAPE and new.tolist() == [4]
    d["lens"] = [bs * d["src"].shape[1] + 1]  # past the tables
    new, ws = run_compact(h, d)
    assert status(ws) == tl.TP_ERR_SHAPE and new.tolist() == d["lens"]


def test_refusals():
    h, h64 = handle(8, 2, 2), handle(8, 2, 2, hd=64)
    L, p = tl.lib(), ctypes.c_void_p(0x10000)
    arr, bad, nul = [(ctypes.c_void_p * 1)(x) for x in (0x10000, 0x10008, None)]

    def copy(hd=h.handle, pairs=p, n=1, layers=1, ck=arr, cv=arr, nb=8, bs=16, ws=p, wb=16):
        return L.tp_kv_cache_copy_blocks(hd, pairs, n, layers, ck, cv, nb, bs, ws, wb, None)
    assert copy(n=0) == tl.TP_OK
    assert copy(hd=h64.handle) == tl.TP_ERR_UNSUPPORTED and copy(n=-1) == tl.TP_ERR_SHAPE
    assert copy(layers=0) == tl.TP_ERR_SHAPE and copy(layers=129) == tl.TP_ERR_UNSUPPORTED
    assert copy(nb=0) == tl.TP_ERR_SHAPE and copy(bs=0) == tl.TP_ERR_SHAPE and copy(nb=1 << 31) == tl.TP_ERR_UNSUPPORTED
    assert copy(pairs=None) == tl.TP_ERR_ARG and copy(pairs=ctypes.c_void_p(0x10004)) == tl.TP_ERR_ARG
    assert copy(ck=None) == tl.TP_ERR_ARG and copy(cv=bad) == tl.TP_ERR_ARG and copy(ck=nul) == tl.TP_ERR_ARG
    assert copy(ws=None) == tl.TP_ERR_ARG and copy(wb=8) == tl.TP_ERR_ARG

    def comp(hd=h.handle, n=1, qsl=p, lens=p, acc=p, m=4, src=p, dst=p, mb=4, layers=1, ck=arr, cv=arr, nb=8, bs=16,
             new=ctypes.c_void_p(0x20000), ws=p, wb=16):
        return L.tp_kv_cache_compact(hd, n, qsl, lens, acc, m, src, dst, mb, layers, ck, cv, nb, bs, new, ws, wb, None)
    assert comp(n=0) == tl.TP_OK
    assert comp(hd=h64.handle) == tl.TP_ERR_UNSUPPORTED and comp(n=-1) == tl.TP_ERR_SHAPE
    assert comp(m=0) == tl.TP_ERR_SHAPE and comp(mb=0) == tl.TP_ERR_SHAPE and comp(layers=0) == tl.TP_ERR_SHAPE
    for k in ("qsl", "lens", "acc", "src", "dst", "new"):
        assert comp(**{k: None}) == tl.TP_ERR_ARG and comp(**{k: ctypes.c_void_p(0x10002)}) == tl.TP_ERR_ARG
    assert comp(new=p) == tl.TP_ERR_ARG                      # the lengths themselves
    assert comp(ws=None) == tl.TP_ERR_ARG
    ck, cv = caches(h, 2, 4, 16, 1)
    with pytest.raises(ValueError):
        h.kv_cache_copy_blocks(dev([(0, 1)]), ck, cv[:1])
    with pytest.raises(ValueError):
        h.kv_cache_copy_blocks(dev([0, 1]), ck, cv)
    with pytest.raises(ValueError):
        h.kv_cache_copy_blocks(dev([(0, 1)]), [ck[0], ck[1][:, :2]], cv)
    with pytest.raises(TypeError):
        h.kv_cache_copy_blocks(dev([(0, 1)]).long(), ck, cv)


def test_refusals_of_caches_that_differ_or_overlap():
    h, L, p = handle(8, 2, 2), tl.lib(), ctypes.c_void_p(0x10000)
    size = 2 * 8 * 16 * 1 * 128 * 2                          # bytes of a cache: t, blocks, block size, kv heads, hd

    def arr(*at):
        return (ctypes.c_void_p * len(at))(*at)

    def both(ck, cv, new=0x20000):
        copy = L.tp_kv_cache_copy_blocks(h.handle, p, 1, len(ck), ck, cv, 8, 16, p, 16, None)
        comp = L.tp_kv_cache_compact(h.handle, 1, p, p, p, 4, p, p, 4, len(ck), ck, cv, 8, 16, ctypes.c_void_p(new), p, 16,
                                     None)
        return copy, comp
    a = 1 << 24
    for ck, cv in [(arr(a), arr(a)), (arr(a, a), arr(a + size, a + 2 * size)),
                   (arr(a, a + 4 * size), arr(a + 2 * size, a + size - 16)), (arr(a + size - 16), arr(a))]:
        assert both(ck, cv) == (tl.TP_ERR_ARG,) * 2 and b"overlap" in L.tp_last_error()
    for new in (0x10000, 0x10004):                           # inside what the call reads
        comp = L.tp_kv_cache_compact(h.handle, 1, ctypes.c_void_p(0x10000), ctypes.c_void_p(0x30000), ctypes.c_void_p(0x40000),
                                     4, ctypes.c_void_p(0x50000), ctypes.c_void_p(0x60000), 4, 1, arr(a), arr(a + size), 8,
                                     16, ctypes.c_void_p(new), p, 16, None)
        assert comp == tl.TP_ERR_ARG and b"new_seq_lens" in L.tp_last_error()
    ck, cv = caches(h, 2, 4, 16, 1)
    pairs = dev([(0, 1)])
    same_bytes = torch.zeros(h.kv_cache_shape(8, 8), dtype=torch.bfloat16, device="cuda")
    for other in (same_bytes, ck[1].view(torch.float16), ck[1].view(torch.int16), ck[1].transpose(1, 2), ck[1].cpu()):
        for k, v in (([ck[0], other], cv), (ck, [cv[0], other])):
            with pytest.raises(ValueError):
                h.kv_cache_copy_blocks(pairs, k, v)
    with pytest.raises(tl.TPError):
        h.kv_cache_copy_blocks(pairs, [ck[0], ck[0]], cv)
