"""Calls on a stream of their own that make their outputs and workspaces themselves, while the caller's current
stream is busy: the results are there when the call's stream is done, and nothing that the caller's stream does
later changes them. (On the CPU: test_streams.py.)
"""
import pytest
import torch

import workloads
import tensor_linear_layers_gb300 as tl
from test_gpu_tree import build, built, check, dev, handle, status  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu

NQ, NKV, SHARDS = 8, 2, 2


@pytest.fixture
def busy():
    """Some 10 ms of copies on the current stream."""
    a, b = (torch.zeros(1 << 30, dtype=torch.uint8, device="cuda") for _ in range(2))

    def start():
        torch.cuda.synchronize()
        for _ in range(32):
            b.copy_(a)
    return start


def test_a_drafted_step_beside_a_busy_stream(busy):
    h = handle(NQ, NKV, SHARDS)
    c = build(NQ, NKV, SHARDS, [1500, 300], [8, 5], 16, seed=150)
    qsl, lens, tables, parents = (dev(x) for x in (c["qsl"], c["lens"], c["tables"], sum(c["parents"], [])))
    qkv, ck, cv = c["qkv"].cuda(), c["ck"].cuda(), c["cv"].cuda()
    st = torch.cuda.Stream()
    for _ in range(3):
        busy()
        mask, pos, mws = tl.tree_mask(parents, qsl, lens, 8, stream=st)
        out, ws = h.tree_attention(qkv, qsl, lens, tables, mask, ck, cv, 8, 1520, stream=st)
        with torch.cuda.stream(st):
            early = out.clone()
        st.synchronize()
        torch.cuda.synchronize()
        assert status(ws) == 0 and status(mws) == 0 and torch.equal(early, out)
        check(out, c, NQ, NKV, SHARDS)
        del mask, pos, mws, out, ws, early                    # their memory goes to the next turn's calls


def test_an_error_status_is_not_wiped(busy):
    h = handle(NQ, NKV, SHARDS)
    st = torch.cuda.Stream()
    busy()
    rope = tl.Rope(64, 128, stream=st)
    qkv = torch.ones(SHARDS, 3, (NQ // SHARDS + 2) * 128, dtype=torch.bfloat16, device="cuda")
    pos, good = dev([1, 64, 2]), dev([1, 63, 2])
    ck = torch.zeros(h.kv_cache_shape(4, 16), dtype=torch.bfloat16, device="cuda")
    cv = torch.zeros_like(ck)
    pairs, qsl, lens, acc, tables = dev([[0, 9]]), dev([0, 3]), dev([10]), dev([[1, 0, -1]]), dev([[0, 1]])
    parents = dev([-1, 1, 0])
    torch.cuda.synchronize()
    busy()
    _, w1 = h.qk_norm_rope(qkv, pos, rope, stream=st)
    w2 = h.kv_cache_copy_blocks(pairs, [ck], [cv], stream=st)
    new, w3 = h.kv_cache_compact(qsl, lens, acc, tables, tables, [ck], [cv], stream=st)
    _, _, w4 = tl.tree_mask(parents, qsl, lens, 3, stream=st)
    out, w5 = h.qk_norm_rope(qkv, good, rope, stream=st)
    st.synchronize()
    torch.cuda.synchronize()
    for w in (w1, w2, w3, w4):
        assert status(w) == tl.TP_ERR_SHAPE
    assert status(w5) == 0 and int(new[0]) == 8
    want, _ = h.qk_norm_rope(qkv, good, tl.Rope(64, 128))
    assert torch.equal(out, want)


def test_captured_on_the_given_stream():
    h = handle(NQ, NKV, SHARDS)
    c = build(NQ, NKV, SHARDS, [700], [8], 16, seed=151)
    qsl, lens, tables, parents = (dev(x) for x in (c["qsl"], c["lens"], c["tables"], sum(c["parents"], [])))
    qkv, ck, cv = c["qkv"].cuda(), c["ck"].cuda(), c["cv"].cuda()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        mask, _, mws = tl.tree_mask(parents, qsl, lens, 8, stream=st)
        out, ws = h.tree_attention(qkv, qsl, lens, tables, mask, ck, cv, 8, 720, stream=st)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert status(ws) == 0 and status(mws) == 0
        check(out, c, NQ, NKV, SHARDS)


def test_blocks_made_and_run_beside_a_busy_stream(busy):
    st, H, inter, T = torch.cuda.Stream(), 256, 512, 40
    w = [workloads.draw(s, 160, i).cuda() for i, s in enumerate([(inter, H), (inter, H), (H, inter)])]
    x = workloads.draw((T, H), 161, 0).cuda()
    cfg = tl.make_config(tl.TP_BLOCK_MLP, 2, H, inter)
    want = tl.TPLinear(cfg, w).mlp_forward(x)["mlp_out"]
    busy()
    blk = tl.TPLinear(cfg, w, stream=st)
    outs = [blk.mlp_forward(x, stream=st)["mlp_out"] for _ in range(3)]
    st.synchronize()
    torch.cuda.synchronize()
    assert status(blk.workspace(T)) == 0 and all(torch.equal(o, want) for o in outs)


def test_paged_attention_beside_a_busy_stream(busy):
    h, st = handle(NQ, NKV, SHARDS), torch.cuda.Stream()
    c = build(NQ, NKV, SHARDS, [1500, 300], [1, 1], 16, seed=152)
    qsl, lens, tables = dev(c["qsl"]), dev(c["lens"]), dev(c["tables"].clip(0))
    qkv, ck, cv = c["qkv"].cuda(), c["ck"].cuda(), c["cv"].cuda()
    busy()
    out, ws = h.paged_attention(qkv, qsl, lens, tables, ck, cv, 1, 1520, stream=st)
    st.synchronize()
    torch.cuda.synchronize()
    assert status(ws) == 0
    check(out, c, NQ, NKV, SHARDS)


@pytest.mark.parametrize("given", [True, False])
def test_moe_routing_arrays_of_other_strides(busy, given):
    T, H, inter, E, k = 37, 256, 512, 4, 2
    w = [workloads.draw(s, 170, i).cuda() for i, s in enumerate([(inter, H), (inter, H), (H, inter)] * E)]
    blk = tl.TPLinear(tl.make_config(tl.TP_BLOCK_MOE, 2, H, inter, n_experts=E), w)
    x = workloads.draw((T, H), 171, 0).cuda()
    rows = torch.arange(T, device="cuda")
    ids = torch.stack([rows % E, (rows // E + 1 + rows) % E]).to(torch.int32)               # [k, T]
    gates = torch.stack([rows.float() / T, 1 - rows.float() / T])
    want = blk.moe_forward(x, ids.t().contiguous(), gates.t().contiguous())
    assert status(blk.workspace(T * k)) == 0
    st = torch.cuda.Stream() if given else None
    busy()
    got = blk.moe_forward(x, ids.t(), gates.t(), stream=st)
    torch.cuda.synchronize()
    assert status(blk.workspace(T * k)) == 0 and torch.equal(got, want)
