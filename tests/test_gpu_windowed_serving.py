"""A windowed model served from paged caches, as a server's steps go: q and k rotated (tp_qk_norm_rope), k and v
written in bf16 (by that call) or in 8 bits (tp_kv_quant_write), attention of everything new (tp_chunk_attention),
o_proj. Prompts in chunks, then steps that mix chunks with decoding requests, then decoding alone, replayed from a
graph. Checked at every step against the float64 oracle on what the steps before put into the cache.
"""
import numpy as np
import pytest
import torch

import oracle
import workloads
import tensor_linear_layers_gb300 as tl
from test_gpu_chunk import check
from test_gpu_kv_quant import built, dev, status  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu

NQ, NKV, T, H, BS, BLOCKS = 8, 2, 2, 256, 16, 80
WINDOW, SINKS = 70, 3
WIDTH = (NQ // T + 2 * NKV // T) * 128


class Server:
    def __init__(self, q8, seed):
        shapes = ((NQ * 128, H), (NKV * 128, H), (NKV * 128, H), (H, NQ * 128))
        self.w = [(workloads.draw(s, seed, i).float() * 0.06).to(torch.bfloat16) for i, s in enumerate(shapes)]
        self.h = tl.TPLinear(tl.make_config(tl.TP_BLOCK_ATTN_PROJ, T, H, n_q_heads=NQ, n_kv_heads=NKV, head_dim=128),
                             [w.cuda() for w in self.w])
        self.rope = tl.Rope(1024, 128, 10000.0)
        self.q8, self.seed, self.steps = q8, seed, 0
        self.lens = [0, 0, 0]
        perm = np.random.default_rng(seed).permutation(BLOCKS)
        self.tables = perm[:3 * 25].reshape(3, 25).astype(np.int32)
        if q8:
            self.cache = self.h.kv_quant_cache(BLOCKS, BS)
        else:
            self.cache = [torch.zeros(self.h.kv_cache_shape(BLOCKS, BS), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        # the caches as the oracle has them
        self.ref = [np.zeros((T, BLOCKS, BS, NKV // T, 128)) for _ in range(2)]
        self.ws = torch.zeros(self.h.chunk_attention_workspace_size(3, 200, 400), dtype=torch.uint8, device="cuda")

    def plan(self, n):
        """Arrays of a step that brings n[b] new tokens of every request."""
        ctx, lens = self.lens, [c + k for c, k in zip(self.lens, n)]
        pos = np.concatenate([np.arange(c, c + k) for c, k in zip(ctx, n)])
        req = np.concatenate([[b] * k for b, k in enumerate(n)]).astype(int)
        slots = self.tables[req, pos // BS] * BS + pos % BS
        x = workloads.draw((len(pos), H), self.seed, 100 + self.steps)
        self.steps += 1
        return dict(x=x, qsl=np.concatenate([[0], np.cumsum(n)]), lens=lens, pos=pos, slots=slots, n=list(n))

    def launch(self, b, max_q, max_len, stream=None):
        """The calls of a step on the GPU's arrays of a plan."""
        h = self.h
        qkv, _ = h.attn_proj_forward(b["x"], None, stream=stream)
        if self.q8:
            rot, w0 = h.qk_norm_rope(qkv, b["pos"], self.rope, out=qkv, stream=stream)
            w1 = h.kv_quant_write(rot, b["slots"], *self.cache, stream=stream)
            sk, sv = self.cache[2:]
        else:
            rot, w0 = h.qk_norm_rope(qkv, b["pos"], self.rope, out=qkv, slot_mapping=b["slots"], cache_k=self.cache[0],
                                     cache_v=self.cache[1], stream=stream)
            w1, sk, sv = w0, None, None
        attn, w2 = h.chunk_attention(rot, b["qsl"], b["lens"], b["tables"], self.cache[0], self.cache[1], max_q, max_len, WINDOW,
                                     SINKS, sk, sv, ws=self.ws, stream=stream)
        _, out = h.attn_proj_forward(None, attn, stream=stream)
        return dict(qkv=rot, attn=attn, out=out, ws=(w0, w1, w2))

    def on_gpu(self, p):
        return {k: (p[k].cuda() if k == "x" else dev(p[k])) for k in ("x", "qsl", "lens", "pos", "slots")} | {"tables": dev(self.tables)}

    def verify(self, p, r):
        assert [status(w) for w in r["ws"]] == [0, 0, 0]
        qkv = r["qkv"].cpu()
        heads = oracle.bf16_to_f64(qkv).reshape(T, len(p["pos"]), -1, 128)
        for which, ref in enumerate(self.ref):
            at = NQ // T + which * (NKV // T)
            new = heads[:, :, at:at + NKV // T]
            new = oracle.values(*oracle.quantise(new)) if self.q8 else new
            ref.reshape(T, -1, NKV // T, 128)[:, p["slots"]] = new
        c = dict(qkv=qkv, qsl=p["qsl"], lens=p["lens"], tables=self.tables, T=len(p["pos"]), bs=BS, heads=(NQ, NKV, T), sk=None,
                 sv=None, ck=torch.from_numpy(self.ref[0]).to(torch.bfloat16), cv=torch.from_numpy(self.ref[1]).to(torch.bfloat16))
        check(r["attn"], c, WINDOW, SINKS)
        # o_proj of what the attention gave
        a = oracle.bf16_to_f64(r["attn"].cpu()).transpose(1, 0, 2).reshape(len(p["pos"]), -1)
        want = a @ oracle.bf16_to_f64(self.w[3]).T
        got = r["out"].double().cpu().numpy()
        assert np.abs(got - want).max() <= 2e-2 * np.abs(want).max()
        self.lens = p["lens"]
        if self.q8:
            k, v, ws = self.h.kv_quant_read(dev(p["slots"]), *self.cache)
            assert status(ws) == 0
            for got, ref in ((k, self.ref[0]), (v, self.ref[1])):
                np.testing.assert_array_equal(got.double().cpu().numpy(), ref.reshape(T, -1, NKV // T, 128)[:, p["slots"]])

    def step(self, n):
        p = self.plan(n)
        self.verify(p, self.launch(self.on_gpu(p), max(n), max(p["lens"])))


@pytest.mark.parametrize("q8", [False, True])
def test_prompts_in_chunks_then_decoding(q8):
    s = Server(q8, 3)
    for n in ([130, 1, 17], [60, 90, 0], [1, 40, 1], [1, 1, 1], [1, 0, 2], [3, 1, 1]):
        s.step(n)
    # decoding steps replayed from a graph: the same buffers, other lengths, slots and tokens at every step
    p = s.plan([1, 1, 1])
    b = s.on_gpu(p)
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        r = s.launch(b, 1, 400, stream=st)
    for k in range(20):
        if k:
            p = s.plan([1, 1, 1])
            for name, x in s.on_gpu(p).items():
                b[name].copy_(x)
        g.replay()
        torch.cuda.synchronize()
        s.verify(p, r)


def test_read_back_into_bf16_pages():
    # an 8-bit cache's tokens read back into bf16 pages: attention over those gives what the codes give, but for how
    # each kernel rounds (both against the same oracle)
    s = Server(True, 5)
    for n in ([150, 20, 40], [1, 1, 60]):
        s.step(n)
    ck, cv = (torch.zeros(s.h.kv_cache_shape(BLOCKS, BS), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = dev(np.arange(BLOCKS * BS))
    k, v, ws = s.h.kv_quant_read(slots, *s.cache)
    assert status(ws) == 0
    ck.view(T, -1, NKV // T, 128)[:] = k
    cv.view(T, -1, NKV // T, 128)[:] = v
    p = s.plan([5, 1, 30])
    r = s.launch(s.on_gpu(p), 30, 400)
    k, v, _ = s.h.kv_quant_read(dev(p["slots"]), *s.cache)
    at = torch.from_numpy(p["slots"]).cuda().long()
    ck.view(T, -1, NKV // T, 128)[:, at] = k
    cv.view(T, -1, NKV // T, 128)[:, at] = v
    out, ws = s.h.chunk_attention(r["qkv"], dev(p["qsl"]), dev(p["lens"]), dev(s.tables), ck, cv, 30, 400, WINDOW, SINKS)
    assert status(ws) == 0
    c = dict(qkv=r["qkv"].cpu(), qsl=p["qsl"], lens=p["lens"], tables=s.tables, T=len(p["pos"]), bs=BS, heads=(NQ, NKV, T), sk=None,
             sv=None, ck=ck.cpu(), cv=cv.cpu())
    check(out, c, WINDOW, SINKS)
    check(r["attn"], c, WINDOW, SINKS)
