"""The calls of a drafted decoding step together, as a server uses them.

A step: the page that holds a request's last tokens is forked (tp_kv_cache_copy_blocks), the drafted
tokens' masks and positions come from their parents (tp_tree_mask), q and k are normed and rotated and
k, v written to the forked pages (tp_qk_norm_rope), the tree attends over them (tp_tree_attention), the
accepted path moves to the request's own pages (tp_kv_cache_compact). The next step goes on from there.
Checked against the float64 oracles on one contiguous sequence, eagerly and replayed from a CUDA graph,
on several streams, and for a layer with rotation bound to it. Attention: max|gpu - ref| <= 2e-2
max|ref| as for the paged attention (k in the cache is rounded once more, to bf16).
"""
import numpy as np
import pytest
import torch

import oracle
import workloads
import tensor_linear_layers_gb300 as tl

pytestmark = pytest.mark.gpu
TOL = 2e-2
f64 = oracle.bf16_to_f64


@pytest.fixture(scope="module", autouse=True)
def built():
    from tensor_linear_layers_gb300 import _build
    _build.build()
    tl.lib()
    torch.cuda.set_device(0)


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def rel(got, ref):
    return float(np.abs(got - ref).max() / max(np.abs(ref).max(), 1e-30))


def handle(nq, nkv, t, H=64):
    cfg = tl.make_config(tl.TP_BLOCK_ATTN_PROJ, t, H, n_q_heads=nq, n_kv_heads=nkv, head_dim=128)
    z = torch.zeros(nq * 128, H, dtype=torch.bfloat16, device="cuda")
    return tl.TPLinear(cfg, [z, z[:nkv * 128].contiguous(), z[:nkv * 128].contiguous(), z.t().contiguous()])


NQ, NKV, T, BS, LAYERS = 8, 2, 2, 16, 3
W = (NQ // T + 2 * NKV // T) * 128


class Server:
    """Two requests, three layers' caches; every token's projected qkv is known ahead (they stand for the model)."""

    def __init__(self, ctx, n, accepted, seed):
        self.h = handle(NQ, NKV, T)
        self.ctx, self.n, self.accepted = list(ctx), n, accepted
        self.gq, self.gk = (workloads.draw((128,), seed, 90 + i, kind="uniform", a=0.5, b=1.5) for i in range(2))
        self.rope = tl.Rope(4096, 128, 10000.0, scaling="yarn", factor=4.0, original_max_position=512,
                            q_gamma=self.gq.cuda(), k_gamma=self.gk.cuda(), eps=1e-5)
        self.freq, self.scale = oracle.rope_frequencies(128, 10000.0, "yarn", 4.0, 512)
        blocks = 64
        self.free = list(np.random.default_rng(seed).permutation(blocks))
        self.ck = [torch.zeros(self.h.kv_cache_shape(blocks, BS), dtype=torch.bfloat16, device="cuda") for _ in range(LAYERS)]
        self.cv = [torch.zeros_like(c) for c in self.ck]
        self.tables = np.zeros((2, 12), dtype=np.int32)
        for b, c in enumerate(ctx):
            for i in range(-(-(c + 40) // BS)):
                self.tables[b, i] = self.free.pop()
        # the prompt of every layer, rotated and written
        self.history = [[workloads.draw((T, c, W), seed, 10 * l + b) for b, c in enumerate(ctx)] for l in range(LAYERS)]
        pos = np.concatenate([np.arange(c) for c in ctx])
        slots = np.concatenate([[self.tables[b, p // BS] * BS + p % BS for p in range(c)] for b, c in enumerate(ctx)])
        for l in range(LAYERS):
            qkv = torch.cat(self.history[l], 1).contiguous().cuda()
            _, ws = self.h.qk_norm_rope(qkv, dev(pos), self.rope, slot_mapping=dev(slots), cache_k=self.ck[l], cache_v=self.cv[l])
            assert int(ws[:4].view(torch.int32)) == 0

    def buffers(self, parents):
        """Static buffers of a step, as a graph would use them."""
        tot = sum(self.n)
        i32 = dict(dtype=torch.int32, device="cuda")
        return dict(
            qkv=[torch.zeros(T, tot, W, dtype=torch.bfloat16, device="cuda") for _ in range(LAYERS)],
            rot=[torch.zeros(T, tot, W, dtype=torch.bfloat16, device="cuda") for _ in range(LAYERS)],
            out=[torch.zeros(T, tot, NQ // T * 128, dtype=torch.bfloat16, device="cuda") for _ in range(LAYERS)],
            parents=dev(parents), qsl=dev(np.concatenate([[0], np.cumsum(self.n)])), lens=torch.zeros(2, **i32),
            pairs=torch.full((4, 2), -1, **i32), slots=torch.zeros(tot, **i32), src=torch.zeros(2, 12, **i32),
            dst=torch.zeros(2, 12, **i32), acc=torch.full((2, 6), -1, **i32), new=torch.zeros(2, **i32),
            mask=torch.zeros(tot, 1, **i32), pos=torch.zeros(tot, **i32), max_len=190,
            ws=torch.zeros(self.h.tree_attention_workspace_size(2, max(self.n), 190), dtype=torch.uint8, device="cuda"))

    def fill(self, s, seed):
        """Host part of a step: forked tables, slots, the drafts' projections."""
        src, pairs, slots = self.tables.copy(), [], []
        for b in range(2):
            for i in range(self.ctx[b] // BS, -(-(self.ctx[b] + self.n[b]) // BS)):
                new = self.free.pop()
                if i == self.ctx[b] // BS and self.ctx[b] % BS:
                    pairs.append((self.tables[b, i], new))
                src[b, i] = new
            slots += [src[b, p // BS] * BS + p % BS for p in range(self.ctx[b], self.ctx[b] + self.n[b])]
        self.drafts = [workloads.draw((T, sum(self.n), W), seed, l) for l in range(LAYERS)]
        for l in range(LAYERS):
            s["qkv"][l].copy_(self.drafts[l])
        s["lens"].copy_(dev([c + n for c, n in zip(self.ctx, self.n)]))
        s["pairs"].fill_(-1)
        s["pairs"][:len(pairs)].copy_(dev(pairs).view(-1, 2) if pairs else s["pairs"][:0])
        s["slots"].copy_(dev(slots))
        s["src"].copy_(dev(src))
        s["dst"].copy_(dev(self.tables))
        s["acc"].fill_(-1)
        for b, a in enumerate(self.accepted):
            s["acc"][b, :len(a)].copy_(dev(a))

    def device(self, s):
        """The step's calls, on the current stream."""
        h = self.h
        h.kv_cache_copy_blocks(s["pairs"], self.ck, self.cv, ws=s["ws"])
        tl.tree_mask(s["parents"], s["qsl"], s["lens"], max(self.n), out=(s["mask"], s["pos"]), ws=s["ws"])
        for l in range(LAYERS):
            h.qk_norm_rope(s["qkv"][l], s["pos"], self.rope, out=s["rot"][l], slot_mapping=s["slots"], cache_k=self.ck[l],
                           cache_v=self.cv[l], ws=s["ws"])
            h.tree_attention(s["rot"][l], s["qsl"], s["lens"], s["src"], s["mask"], self.ck[l], self.cv[l], max(self.n),
                             s["max_len"], out=s["out"][l], ws=s["ws"])
        h.kv_cache_compact(s["qsl"], s["lens"], s["acc"], s["src"], s["dst"], self.ck, self.cv, out=s["new"], ws=s["ws"])

    def rotated(self, qkv, pos):
        return oracle.qk_norm_rope(qkv, pos, self.freq, NQ, NKV, 128, T, False, self.scale, self.gq, self.gk, 1e-5)

    def check(self, s, parents):
        """Every drafted token against the contiguous sequence of its path; then the accepted ones become history."""
        assert int(s["ws"][:4].view(torch.int32)) == 0
        at = 0
        for b in range(2):
            par, c = parents[at:at + self.n[b]], self.ctx[b]
            sees = oracle.tree_sees(par)
            for l in range(LAYERS):
                for i in range(self.n[b]):
                    path = np.nonzero(sees[i])[0]
                    seq = torch.cat([self.history[l][b], self.drafts[l][:, at + path]], 1)
                    rot = self.rotated(seq, np.arange(c + len(path)))
                    ref = oracle.attention_rows(rot, NQ, NKV, 128, T, [0, c + len(path)], [c + len(path) - 1])
                    assert rel(f64(s["out"][l][:, at + i].cpu()), ref[:, 0]) <= TOL
                self.history[l][b] = torch.cat([self.history[l][b], self.drafts[l][:, [at + a for a in self.accepted[b]]]], 1)
            self.ctx[b] += len(self.accepted[b])
            at += self.n[b]
        assert s["new"].tolist() == self.ctx


PARENTS = [-1, 0, 0, 1, 2, -1, 5] + [-1, 0, 1, 1, 3]
N, ACCEPTED = [7, 5], [[0, 2, 4], [0, 1, 3, 4]]


@pytest.mark.parametrize("graph", [False, True])
def test_steps_follow_each_other(graph):
    sv = Server([37, 16], N, ACCEPTED, seed=3)
    s = sv.buffers(PARENTS)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        if graph:
            sv.fill(s, 99)
            keep = [c.clone() for c in sv.ck + sv.cv]
            sv.device(s)                                # a first pass outside the capture
            st.synchronize()
            for c, k in zip(sv.ck + sv.cv, keep):
                c.copy_(k)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=st):
                sv.device(s)
        for step in range(3):
            sv.fill(s, 100 + step)
            if graph:
                g.replay()
            else:
                sv.device(s)
            st.synchronize()
            sv.check(s, PARENTS)


FIRST_CALLS_CAPTURED = """
import sys
sys.path.insert(0, {root!r})
import torch
from tests import test_gpu_draft_step as m
import tensor_linear_layers_gb300 as tl
h = m.handle(m.NQ, m.NKV, m.T)
rope = tl.Rope(512, 128)
blocks, n, ctx = 16, 5, 40
ck = [torch.randn(h.kv_cache_shape(blocks, m.BS), device="cuda").to(torch.bfloat16) for _ in range(2)]
cv = [torch.randn(h.kv_cache_shape(blocks, m.BS), device="cuda").to(torch.bfloat16) for _ in range(2)]
src = torch.randn(m.T, n, m.W, device="cuda").to(torch.bfloat16)
qkv, rot = torch.zeros_like(src), torch.zeros_like(src)
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
parents, qsl, lens, tab = i32([-1, 0, 0, 1, 2]), i32([0, n]), i32([ctx + n]), i32([[3, 1, 4, 9]])
pairs, acc, new = i32([[4, 12]]), i32([[0, 2, 4]]), i32([0])
slots = i32([(ctx + j) % 16 + 16 * [3, 1, 4, 9][(ctx + j) // 16] for j in range(n)])
mask, pos = torch.zeros(n, 1, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
out = torch.zeros(m.T, n, m.NQ // m.T * 128, dtype=torch.bfloat16, device="cuda")
ws = torch.zeros(h.tree_attention_workspace_size(1, n, 64), dtype=torch.uint8, device="cuda")

def step():
    qkv.copy_(src)                       # a copy node in front of a programmatic launch
    h.kv_cache_copy_blocks(pairs, ck, cv, ws=ws)
    tl.tree_mask(parents, qsl, lens, n, out=(mask, pos), ws=ws)
    h.qk_norm_rope(qkv, pos, rope, out=rot, slot_mapping=slots, cache_k=ck[0], cache_v=cv[0], ws=ws)
    out.zero_()                          # a memset node
    h.tree_attention(rot, qsl, lens, tab, mask, ck[0], cv[0], n, 64, out=out, ws=ws)
    h.kv_cache_compact(qsl, lens, acc, tab, tab, ck, cv, out=new, ws=ws)

keep = [x.clone() for x in ck + cv]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    step()
g.replay()
torch.cuda.synchronize()
assert int(ws[:4].view(torch.int32)) == 0 and new.tolist() == [ctx + 3]
a = [out.clone(), rot.clone(), mask.clone(), pos.clone()] + [x.clone() for x in ck + cv]
for x, k in zip(ck + cv, keep):
    x.copy_(k)
step()
torch.cuda.synchronize()
for x, y in zip(a, [out, rot, mask, pos] + ck + cv):
    assert torch.equal(x, y)
print("captured first: ok")
"""


def test_calls_captured_before_they_ever_ran_and_after_copies():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED.format(root=root)], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "captured first: ok" in r.stdout, r.stdout + r.stderr


def test_two_streams_with_their_own_workspaces():
    a, b = Server([37, 16], N, ACCEPTED, seed=3), Server([50, 90], N, ACCEPTED, seed=4)
    sa, sb = a.buffers(PARENTS), b.buffers(PARENTS)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    a.fill(sa, 7)
    b.fill(sb, 8)
    torch.cuda.synchronize()
    for _ in range(3):                                  # the same step again: it reads and writes the same places
        for srv, s, st in ((a, sa, streams[0]), (b, sb, streams[1])):
            with torch.cuda.stream(st):
                srv.device(s)
    torch.cuda.synchronize()
    a.check(sa, PARENTS)
    b.check(sb, PARENTS)


def test_stream_argument():
    sv = Server([37, 16], N, ACCEPTED, seed=3)
    s = sv.buffers(PARENTS)
    sv.fill(s, 7)
    sv.device(s)
    torch.cuda.synchronize()
    want = [o.clone() for o in s["out"]]
    st = torch.cuda.Stream()
    out = torch.zeros_like(want[0])
    tl.tree_mask(s["parents"], s["qsl"], s["lens"], max(N), out=(s["mask"], s["pos"]), ws=s["ws"], stream=st)
    sv.h.qk_norm_rope(s["qkv"][0], s["pos"], sv.rope, out=s["rot"][0], ws=s["ws"], stream=st)
    sv.h.tree_attention(s["rot"][0], s["qsl"], s["lens"], s["src"], s["mask"], sv.ck[0], sv.cv[0], max(N), 190, out=out,
                        ws=s["ws"], stream=st)
    st.synchronize()
    assert torch.equal(out, want[0])


def test_paged_decode_after_rotation_matches_the_contiguous_sequence():
    # one new token per request through the rotation (which writes the cache) and the ordinary paged attention
    sv = Server([37, 80], [1, 1], [[0], [0]], seed=5)
    new = [workloads.draw((T, 2, W), 55, 0)]
    pos = np.array(sv.ctx)
    slots = [sv.tables[b, p // BS] * BS + p % BS for b, p in enumerate(pos)]
    rot, ws = sv.h.qk_norm_rope(new[0].cuda(), dev(pos), sv.rope, slot_mapping=dev(slots), cache_k=sv.ck[0], cache_v=sv.cv[0])
    out, ws2 = sv.h.paged_attention(rot, dev([0, 1, 2]), dev(pos + 1), dev(sv.tables), sv.ck[0], sv.cv[0], 1, 81)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32)) == 0 and int(ws2[:4].view(torch.int32)) == 0
    for b in range(2):
        seq = torch.cat([sv.history[0][b], new[0][:, b:b + 1]], 1)
        r = sv.rotated(seq, np.arange(pos[b] + 1))
        ref = oracle.attention_rows(r, NQ, NKV, 128, T, [0, pos[b] + 1], [pos[b]])
        assert rel(f64(out[:, b].cpu()), ref[:, 0]) <= TOL


@pytest.mark.parametrize("gathered", [False, True])
def test_layer_with_rotation(gathered):
    w = workloads.Workload("case", "layer", T=200, H=256, I=512, nq=4, nkv=2, hd=128, t=2, w_std=0.02, norm=True, seed=1)
    d = workloads.layer_inputs(w)
    fl = tl.TP_FLAG_HAS_NORM | (tl.TP_FLAG_GATHERED if gathered else 0)
    ca = tl.make_config(tl.TP_BLOCK_ATTN_PROJ, w.t, w.H, n_q_heads=w.nq, n_kv_heads=w.nkv, head_dim=w.hd, flags=fl)
    cm = tl.make_config(tl.TP_BLOCK_MLP, w.t, w.H, w.I, flags=fl)
    attn = tl.TPLinear(ca, [d[k].cuda() for k in ("w_q", "w_k", "w_v", "w_o")], gamma=d["gamma_attn"].cuda())
    mlp = tl.TPLinear(cm, [d[k].cuda() for k in ("w_gate", "w_up", "w_down")], gamma=d["gamma_mlp"].cuda())
    layer = tl.TPLayer(attn, mlp, 256)
    cu = [0, 120, 200]
    args = (d["hidden"].cuda(), d["residual"].cuda(), dev(cu), 120)
    plain = {k: v.clone() for k, v in layer.forward(*args).items()}
    gq, gk = (workloads.draw((128,), 9, i, kind="uniform", a=0.5, b=1.5) for i in range(2))
    rope = tl.Rope(512, 64, 10000.0, layout=tl.TP_ROPE_INTERLEAVED, q_gamma=gq.cuda(), k_gamma=gk.cuda(), eps=1e-5)
    pos = np.concatenate([np.arange(120), 30 + np.arange(80), np.zeros(56)])
    layer.set_rope(rope, dev(pos))
    out = layer.forward(*args)
    torch.cuda.synchronize()
    assert int(layer.workspace()[:4].view(torch.int32)) == 0
    # the same steps through the separate calls: the same bits
    x1, _ = tl.add_rms_norm(args[0], args[1], attn.gamma, 1e-5)
    qkv, _ = attn.attn_proj_forward(x1, None)
    attn.qk_norm_rope(qkv, dev(pos), rope, out=qkv)
    a = attn.attention_forward(qkv, args[2], 120)
    _, o = attn.attn_proj_forward(None, a)
    assert torch.equal(o, out["attn_out"])
    # and the oracle: projections of the oracle's own norm, rotated, attended, projected
    f, _ = oracle.rope_frequencies(64, 10000.0)
    n64, _ = oracle.add_rms_norm(f64(d["hidden"]), f64(d["residual"]), f64(d["gamma_attn"]), 1e-5)
    q64 = oracle.qkv_parallel(n64, f64(d["w_q"]), f64(d["w_k"]), f64(d["w_v"]), w.nq, w.nkv, w.hd, w.t)
    r64 = oracle.qk_norm_rope(q64, pos[:200], f, w.nq, w.nkv, w.hd, w.t, True, 1.0, gq, gk, 1e-5)
    a64 = oracle.attention_core(r64, w.nq, w.nkv, w.hd, w.t, cu)
    ref = oracle.o_proj_parallel(a64, f64(d["w_o"]), w.t)
    assert rel(f64(out["attn_out"].cpu()), ref) <= TOL
    # a position past the table is reported; without rotation the layer is as before
    layer.set_rope(rope, dev(np.full(256, 512)))
    layer.forward(*args)
    torch.cuda.synchronize()
    assert int(layer.workspace()[:4].view(torch.int32)) == tl.TP_ERR_SHAPE
    layer.workspace().zero_()
    layer.set_rope(None)
    again = layer.forward(*args)
    torch.cuda.synchronize()
    assert all(torch.equal(again[k], plain[k]) for k in plain)
    with pytest.raises(ValueError):
        layer.set_rope(rope)
    with pytest.raises(ValueError):
        layer.set_rope(rope, dev(pos[:200]))
