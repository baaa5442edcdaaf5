"""One tree-attention workspace over calls of other lengths, under bounds well above them (a server's fixed
max_seq_len, a captured graph), against the float64 oracle with the tolerance of test_gpu_tree.py.

The work split then gives a CTA fewer places than a chunk takes unless it is held to one, and the merge would
read slots that the call did not write: an earlier call's. The tests fill everything behind the status word with
NaN before the call, or run a longer call on it first.
"""
import numpy as np
import pytest
import torch

import tensor_linear_layers_gb300 as tl
from test_gpu_tree import build, built, check, dev, handle, run, status  # noqa: F401 (built: the module's fixture)

pytestmark = pytest.mark.gpu

NQ, NKV, T_SHARDS = 32, 8, 4


def workspace(h, reqs, max_q, max_len, fill=None):
    ws = torch.zeros(h.tree_attention_workspace_size(reqs, max_q, max_len), dtype=torch.uint8, device="cuda")
    if fill is not None:
        ws[256:] = fill                                       # 0xff: NaN in every partial result
    return ws


CALLS = [  # bounds (max_query_len, max_seq_len), then the calls' cached and drafted tokens
    (8, 8192, [([1492], [8]), ([692], [8])]),
    (8, 8192, [([2392], [8]), ([1292], [8])]),
    (8, 1000, [([992, 492], [8, 8]), ([592, 392], [8, 8])]),
    (8, 900, [([892, 12, 0, 300, 120, 511], [8, 8, 5, 1, 8, 3]), ([12, 700, 250, 0, 380, 90], [8, 8, 1, 8, 6, 8])]),
    (64, 8192, [([1460, 250], [40, 8]), ([660, 100], [40, 8])]),          # tiles of one and of two times 128 rows
    (64, 4096, [([700], [8]), ([300], [8]), ([1500], [64])]),             # the kernel of two tiles for one tile's rows
    (256, 2048, [([600], [256]), ([120, 70], [100, 33])]),                # groups of 256 rows
]


@pytest.mark.parametrize("max_q,max_len,calls", CALLS)
def test_calls_of_other_lengths_on_one_workspace(max_q, max_len, calls):
    h = handle(NQ, NKV, T_SHARDS)
    ws = workspace(h, max(len(c) for c, _ in calls), max_q, max_len)
    for i, (ctx, n) in enumerate(calls + calls[:1]):
        c = build(NQ, NKV, T_SHARDS, ctx, n, 16, seed=70 + i)
        c["tables"] = np.pad(c["tables"], ((0, 0), (0, -(-max_len // 16) + 1 - c["tables"].shape[1])), constant_values=-5)
        out, _ = run(h, c, max_q=max_q, max_len=max_len, ws=ws)
        assert status(ws) == 0
        check(out, c, NQ, NKV, T_SHARDS)


@pytest.mark.parametrize("max_q,max_len,calls", CALLS)
@pytest.mark.parametrize("fill", [0xff, 0xc2])                # NaN and -97.4 in every partial value
def test_nothing_but_this_calls_results_is_merged(max_q, max_len, calls, fill):
    h = handle(NQ, NKV, T_SHARDS)
    for ctx, n in calls:
        c = build(NQ, NKV, T_SHARDS, ctx, n, 16, seed=80 + len(n))
        c["tables"] = np.pad(c["tables"], ((0, 0), (0, -(-max_len // 16) + 1 - c["tables"].shape[1])), constant_values=-5)
        clean, _ = run(h, c, max_q=max_q, max_len=max_len, ws=workspace(h, len(ctx), max_q, max_len))
        got, ws = run(h, c, max_q=max_q, max_len=max_len, ws=workspace(h, len(ctx), max_q, max_len, fill))
        assert status(ws) == 0 and torch.equal(got, clean)


def test_scores_far_below_zero_under_a_wide_bound():
    # every score of a row near -300: a slot of zeros taken for a part would have the row's largest score
    h = handle(8, 2, 2)
    c = build(8, 2, 2, [1000], [3], 16, seed=91)
    c["qkv"].zero_()
    c["qkv"][:, :, :4 * 128:128] = 16.0                       # q heads (16, 0, 0, ..): the score is k's first element
    c["ck"][..., 0] = (-208.0 + c["ck"][..., 0].float().clamp(-2, 2)).to(torch.bfloat16)     # times 16 / sqrt(128)
    c["tables"] = np.pad(c["tables"], ((0, 0), (0, 600 - c["tables"].shape[1])), constant_values=-5)
    out, ws = run(h, c, max_q=8, max_len=8192)
    assert status(ws) == 0
    check(out, c, 8, 2, 2)


@pytest.mark.parametrize("max_q,max_len,lens", [(8, 8192, (1500, 700, 130, 2400)), (64, 8192, (1500, 300, 900))])
def test_a_captured_call_replayed_for_other_lengths(max_q, max_len, lens):
    h = handle(NQ, NKV, T_SHARDS)
    n = [8, 5]
    cases = [build(NQ, NKV, T_SHARDS, [L - 8, L // 2], n, 16, seed=100 + i) for i, L in enumerate(lens)]
    blocks = max(c["ck"].shape[1] for c in cases)
    pad = torch.nn.functional.pad
    mb = max_len // 16
    s = dict(qkv=torch.zeros_like(cases[0]["qkv"]).cuda(), lens=dev([8, 5]), qsl=dev([0, 8, 13]),
             tables=torch.full((2, mb), -5, dtype=torch.int32, device="cuda"), parents=dev([-1] * 13),
             ck=torch.zeros(T_SHARDS, blocks, *cases[0]["ck"].shape[2:], dtype=torch.bfloat16, device="cuda"))
    s["cv"] = torch.zeros_like(s["ck"])
    ws = workspace(h, 2, max_q, max_len)
    out = torch.empty(T_SHARDS, 13, NQ // T_SHARDS * 128, dtype=torch.bfloat16, device="cuda")
    mask = torch.empty(13, -(-max_q // 32), dtype=torch.int32, device="cuda")
    pos = torch.empty(13, dtype=torch.int32, device="cuda")

    def load(c):
        s["qkv"].copy_(c["qkv"])
        s["lens"].copy_(dev(c["lens"]))
        t = torch.full((2, mb), -5, dtype=torch.int32)
        t[:, :c["tables"].shape[1]] = torch.from_numpy(c["tables"][:, :mb])
        s["tables"].copy_(t)
        s["parents"].copy_(dev(sum(c["parents"], [])))
        for k in ("ck", "cv"):
            s[k].copy_(pad(c[k], (0, 0, 0, 0, 0, 0, 0, blocks - c[k].shape[1])))

    def step():
        tl.tree_mask(s["parents"], s["qsl"], s["lens"], max_q, out=(mask, pos), ws=ws)
        h.tree_attention(s["qkv"], s["qsl"], s["lens"], s["tables"], mask, s["ck"], s["cv"], max_q, max_len, out=out, ws=ws)

    load(cases[0])
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for c in cases + cases[:1]:
        load(c)
        g.replay()
        torch.cuda.synchronize()
        assert status(ws) == 0
        check(out, c, NQ, NKV, T_SHARDS)
