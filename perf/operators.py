"""Cases that measure the operators of a speculative decoding step on a paged KV cache.

Four operators, each in its plain form (elementary torch operations in 32 bits) and as the framework's call:

* ``rope``     per-head RMSNorm of q and k (optional) and rotary positions, k and v written to their cache slots
* ``tree``     attention of a tree of drafted tokens over the paged cache (ancestor masks and positions from the
               tree's parent indices included)
* ``fork``     copies of cache pages, all layers in one call
* ``compact``  the accepted tokens of every request moved from the pages that held the drafts to the request's own
               pages, all layers in one call

Layouts are the framework's: qkv [t][T][q heads | k heads | v heads of the shard][128], caches
[t][blocks][block_size][kv heads of the shard][128], all bf16.
"""
import math

import torch

own = False

HD = 128
DEV = "cuda"


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of 32 requests at far positions, frequencies scaled in bands for a long context
        {"name": "rope_decode", "op": "rope", "T": 32, "nq": 32, "nkv": 8, "t": 4, "rd": 128, "half": True,
         "norm": False, "scaling": "bands", "max_pos": 131072, "bs": 16, "write": True},
        # prefill of a model that norms its q and k heads, cache written
        {"name": "norm_rope_prefill", "op": "rope", "T": 4096, "nq": 32, "nkv": 8, "t": 4, "rd": 128, "half": True,
         "norm": True, "scaling": "none", "max_pos": 4096, "bs": 16, "write": True},
        # ragged batch, half of each head rotated in adjacent pairs, far positions, no cache (feeds the attention core)
        {"name": "norm_rope_partial", "op": "rope", "T": 2043, "nq": 28, "nkv": 4, "t": 4, "rd": 64, "half": False,
         "norm": True, "scaling": "yarn", "max_pos": 65536, "bs": 16, "write": False},
        # the widest prefill: 64 q heads, 8192 tokens
        {"name": "rope_prefill_wide", "op": "rope", "T": 8192, "nq": 64, "nkv": 8, "t": 8, "rd": 128, "half": True,
         "norm": False, "scaling": "bands", "max_pos": 16384, "bs": 32, "write": True},
        # one user, a small tree over a short context: latency
        {"name": "tree_single", "op": "tree", "reqs": 1, "n": 8, "ctx_lo": 500, "ctx_hi": 500, "nq": 32, "nkv": 8,
         "t": 4, "bs": 16},
        # the decode batch of 32 requests with up to 8 drafted tokens each
        {"name": "tree_batch", "op": "tree", "reqs": 32, "n": 8, "ctx_lo": 248, "ctx_hi": 4088, "nq": 32, "nkv": 8,
         "t": 4, "bs": 16},
        # large trees (up to 64 tokens) and groups of 7 q heads: matrix products bound it
        {"name": "tree_wide", "op": "tree", "reqs": 32, "n": 64, "ctx_lo": 1024, "ctx_hi": 8100, "nq": 28, "nkv": 4,
         "t": 4, "bs": 32},
        # two long documents, 26 drafted tokens each
        {"name": "tree_long", "op": "tree", "reqs": 2, "n": 26, "ctx_lo": 130001, "ctx_hi": 131040, "nq": 64,
         "nkv": 8, "t": 8, "bs": 64},
        # a few requests fork their last page, all layers
        {"name": "fork_few", "op": "fork", "pairs": 4, "blocks": 64, "layers": 32, "nq": 32, "nkv": 8, "t": 4,
         "bs": 16},
        # a batch of forks
        {"name": "fork_many", "op": "fork", "pairs": 96, "blocks": 400, "layers": 32, "nq": 32, "nkv": 8, "t": 4,
         "bs": 16},
        # one user's accepted path, all layers
        {"name": "compact_single", "op": "compact", "reqs": 1, "n": 8, "acc": 5, "ctx_lo": 203, "ctx_hi": 203,
         "layers": 32, "nq": 32, "nkv": 8, "t": 4, "bs": 16},
        # the accepted paths of 64 requests with 32 drafted tokens each
        {"name": "compact_batch", "op": "compact", "reqs": 64, "n": 32, "acc": 9, "ctx_lo": 17, "ctx_hi": 120,
         "layers": 32, "nq": 64, "nkv": 8, "t": 8, "bs": 16},
    ]


HEADS = ((32, 8), (28, 4), (64, 8), (8, 2), (4, 4))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    nq, nkv = rng.choice(HEADS)
    t = rng.choice([t for t in (1, 2, 4, 8) if nq % t == 0 and (nkv % t == 0 or t % nkv == 0)])
    return {"nq": nq, "nkv": nkv, "t": t}


def draw(rng):
    op = rng.choice(("rope", "rope", "tree", "tree", "tree", "fork", "compact"))
    c = {"op": op, **_heads(rng)}
    if op == "rope":
        c.update(T=_log(rng, 1, 8192), rd=rng.choice((128, 128, 64, 32, 96, 20)), half=rng.random() < 0.6,
                 norm=rng.random() < 0.5, scaling=rng.choice(("none", "linear", "ntk", "bands", "yarn")),
                 max_pos=_log(rng, 8192, 131072), bs=rng.choice((1, 16, 24, 32, 64)), write=rng.random() < 0.7)
    elif op == "tree":
        reqs = _log(rng, 1, 48)
        n = _log(rng, 1, 64)
        # the cached keys of all requests and the products of all queries stay within the largest listed case's
        kv = max(c["nkv"], c["t"])
        most = min(2 * 130000 * 8 // (reqs * kv), 2 * 130000 * 26 * 64 // (reqs * n * c["nq"]), 120000)
        hi = _log(rng, 16, max(17, most))
        c.update(reqs=reqs, n=n, ctx_lo=rng.randint(0, hi), ctx_hi=hi, bs=rng.choice((1, 8, 16, 24, 32, 64, 128)))
    elif op == "fork":
        layers = _log(rng, 1, 48)
        bs = rng.choice((1, 16, 24, 32))
        pairs = _log(rng, 1, min(512, max(2, 96 * 32 * 16 * 8 // (layers * bs * max(c["nkv"], c["t"]) * 2))))
        c.update(pairs=pairs, blocks=2 * pairs + rng.randint(1, 20), layers=layers, bs=bs)
    else:
        reqs = _log(rng, 1, 64)
        n = _log(rng, 1, 48)
        lo = rng.randint(0, 100)
        c.update(reqs=reqs, n=n, acc=rng.randint(1, min(9, n)), ctx_lo=lo, ctx_hi=lo + rng.randint(0, 20),
                 layers=_log(rng, 1, 32), bs=rng.choice((1, 8, 16, 24, 32)))
    return c


# ---------------------------------------------------------------------------------------------- shapes
def _shape(c):
    q_per = c["nq"] // c["t"]
    kv_per = 1 if c["t"] >= c["nkv"] else c["nkv"] // c["t"]
    return q_per, kv_per, (q_per + 2 * kv_per) * HD


def _spread(n, lo, hi):
    """n whole numbers of [lo, hi], spread evenly in an irregular order (the case alone fixes them)."""
    return [lo + int((hi - lo + 1) * ((0.381966 + 0.618034 * i) % 1.0)) for i in range(n)]


def _tree_sizes(c):
    """Cached tokens and drafted tokens of each request."""
    n = [c["n"]] * c["reqs"] if c["reqs"] <= 2 else _spread(c["reqs"], max(1, c["n"] // 2), c["n"])
    return _spread(c["reqs"], c["ctx_lo"], c["ctx_hi"]), n


def _accepted(c):
    return [c["acc"]] if c["reqs"] == 1 else [min(a, n) for a, n in zip(_spread(c["reqs"], 0, c["acc"]), _tree_sizes(c)[1])]


def work(c):
    q_per, kv_per, w = _shape(c)
    t = c["t"]
    if c["op"] == "rope":
        b = 2 * c["T"] * t * w * 2 + c["T"] * (c["rd"] * 4 + 4)
        if c["write"]:
            b += 2 * c["T"] * t * kv_per * HD * 2 + 4 * c["T"]
        return {"bytes": b, "flops": 8.0 * c["T"] * t * (q_per + kv_per) * HD}
    if c["op"] == "tree":
        ctx, n = _tree_sizes(c)
        keys = sum(x + k for x, k in zip(ctx, n))
        T = sum(n)
        b = keys * t * kv_per * HD * 4 + 2 * T * t * q_per * HD * 2
        b += sum(4 * (-(-(x + k) // c["bs"])) for x, k in zip(ctx, n)) + T * (8 + 4 * (-(-c["n"] // 32)))
        return {"bytes": b, "flops": 4.0 * HD * c["nq"] * sum(k * (x + k) for x, k in zip(ctx, n))}
    if c["op"] == "fork":
        return {"bytes": 2 * c["pairs"] * c["layers"] * 2 * t * c["bs"] * kv_per * HD * 2 + 8 * c["pairs"], "flops": 0}
    moved = sum(_accepted(c))
    return {"bytes": 2 * moved * c["layers"] * 2 * t * kv_per * HD * 2 + 4 * (moved + 4 * c["reqs"]), "flops": 0}


# ---------------------------------------------------------------------------------------------- inputs
ROPE_BASE, ROPE_FACTOR, ROPE_ORIGINAL = 500000.0, 8.0, 8192
LOW_FREQ, HIGH_FREQ = 1.0, 4.0         # of the bands scaling
BETA_SLOW, BETA_FAST = 1.0, 32.0       # of the yarn scaling
EPS = 1e-6


def _handle(c):
    """The framework's attention handle of these head counts (its projections are not used here)."""
    import tensor_linear_layers_gb300 as tl
    cfg = tl.make_config(tl.TP_BLOCK_ATTN_PROJ, c["t"], 256, n_q_heads=c["nq"], n_kv_heads=c["nkv"], head_dim=HD)
    z = torch.zeros(c["nq"] * HD * 256, dtype=torch.bfloat16, device=DEV)
    kv = z[:c["nkv"] * HD * 256].view(-1, 256)
    return tl.TPLinear(cfg, [z.view(-1, 256), kv, kv, z.view(256, -1)])


def _tables(g, lens, bs, extra=3):
    """Block tables [n, max blocks] of scattered pages for these token counts, and the number of pages."""
    need = [-(-n // bs) for n in lens]
    blocks = sum(need) + extra
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    cols = max(max(need), 1)
    first = torch.tensor([sum(need[:b]) for b in range(len(need))], device=DEV)
    at = first[:, None] + torch.arange(cols, device=DEV)
    return perm[at.clamp(max=blocks - 1)].contiguous(), blocks


def _yarn_mscale():
    return 0.1 * math.log(ROPE_FACTOR) + 1.0


def _inv_freq(c):
    """Angle per position of each rotated pair, in 64 bits."""
    rd = c["rd"]
    i = torch.arange(0, rd, 2, dtype=torch.float64, device=DEV)
    kind = c["scaling"]
    base = ROPE_BASE * ROPE_FACTOR ** (rd / (rd - 2)) if kind == "ntk" else ROPE_BASE
    f = base ** (-i / rd)
    if kind == "linear":
        f = f / ROPE_FACTOR
    elif kind == "bands":
        turns = ROPE_ORIGINAL * f / (2 * math.pi)
        mix = ((turns - LOW_FREQ) / (HIGH_FREQ - LOW_FREQ)).clamp(0, 1)
        f = f / ROPE_FACTOR * (1 - mix) + f * mix
    elif kind == "yarn":
        at = [rd * math.log(ROPE_ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(ROPE_BASE))
              for turns in (BETA_FAST, BETA_SLOW)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rd - 1)
        ramp = ((i / 2 - lo) / (hi - lo if hi > lo else 0.001)).clamp(0, 1)
        f = f / ROPE_FACTOR * ramp + f * (1 - ramp)
    return f


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    q_per, kv_per, w = _shape(c)
    t = c["t"]
    s = {"c": c}

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)

    def ints(lo, hi, n):
        return torch.randint(lo, hi, (n,), generator=g, device=DEV)

    if own:
        s["blk"] = _handle(c)
    if c["op"] == "rope":
        T = c["T"]
        s["qkv"] = normal(t, T, w)
        # decode: each token anywhere; prefill: consecutive positions from a random start
        far, start = ints(0, c["max_pos"], T), ints(0, c["max_pos"], 1)
        s["pos"] = (far if T <= 256 else (start + torch.arange(T, device=DEV)) % c["max_pos"]).to(torch.int32)
        s["gq"] = s["gk"] = None
        if c["norm"]:
            s["gq"], s["gk"] = (1 + 0.2 * normal(HD)), (1 + 0.2 * normal(HD))
        if own:
            import tensor_linear_layers_gb300 as tl
            s["rope"] = tl.Rope(c["max_pos"], c["rd"], ROPE_BASE,
                                layout=tl.TP_ROPE_HALF if c["half"] else tl.TP_ROPE_INTERLEAVED,
                                scaling=c["scaling"], factor=ROPE_FACTOR, original_max_position=ROPE_ORIGINAL,
                                low_freq_factor=LOW_FREQ, high_freq_factor=HIGH_FREQ, beta_slow=BETA_SLOW,
                                beta_fast=BETA_FAST, q_gamma=s["gq"], k_gamma=s["gk"], eps=EPS, device=DEV)
        else:
            angle = torch.arange(c["max_pos"], dtype=torch.float64, device=DEV)[:, None] * _inv_freq(c)
            m = _yarn_mscale() if c["scaling"] == "yarn" else 1.0
            s["cos"], s["sin"] = (angle.cos() * m).float(), (angle.sin() * m).float()
        s["out"] = torch.empty_like(s["qkv"])
        s["ws"] = torch.zeros(16, dtype=torch.uint8, device=DEV)
        s["slots"] = s["ck"] = s["cv"] = None
        if c["write"]:
            blocks = -(-T // c["bs"]) + 4
            s["slots"] = torch.randperm(blocks * c["bs"], generator=g, device=DEV)[:T].to(torch.int32)
            s["ck"], s["cv"] = (normal(t, blocks, c["bs"], kv_per, HD) for _ in range(2))
        return s
    if c["op"] == "fork":
        s["ck"], s["cv"] = (normal(c["layers"], t, c["blocks"], c["bs"], kv_per, HD) for _ in range(2))
        perm = torch.randperm(c["blocks"], generator=g, device=DEV)
        # a page may be forked several times; the targets are free pages
        src = perm[c["pairs"]:][ints(0, c["blocks"] - c["pairs"], c["pairs"])]
        s["pairs"] = torch.stack([src, perm[:c["pairs"]]], 1).to(torch.int32).contiguous()
        s["ws"] = torch.zeros(16, dtype=torch.uint8, device=DEV)
        s["lk"], s["lv"] = list(s["ck"].unbind(0)), list(s["cv"].unbind(0))
        return s
    ctx, n = _tree_sizes(c)
    lens = [x + k for x, k in zip(ctx, n)]
    s["n"], s["max_len"] = max(n), max(lens)
    s["qsl"] = torch.tensor([sum(n[:b]) for b in range(len(n) + 1)], dtype=torch.int32, device=DEV)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["tables"], blocks = _tables(g, lens, c["bs"])
    if c["op"] == "tree":
        s["qkv"] = normal(t, sum(n), w) * 1.5
        s["ck"], s["cv"] = (normal(t, blocks, c["bs"], kv_per, HD) for _ in range(2))
        # each drafted token's parent: one of the few before it, or the last cached token (-1)
        i = torch.cat([torch.arange(k, device=DEV) for k in n])
        back = 1 + (torch.rand(len(i), generator=g, device=DEV) * 4).long()
        s["parents"] = (i - back).clamp(min=-1).to(torch.int32)
        s["words"] = -(-s["n"] // 32)
        s["mask"] = torch.empty(sum(n), s["words"], dtype=torch.int32, device=DEV)
        s["pos"] = torch.empty(sum(n), dtype=torch.int32, device=DEV)
        s["out"] = torch.empty(t, sum(n), q_per * HD, dtype=torch.bfloat16, device=DEV)
        if own:
            size = s["blk"].tree_attention_workspace_size(c["reqs"], s["n"], s["max_len"])
            s["ws"] = torch.zeros(size, dtype=torch.uint8, device=DEV)
        return s
    # compact: the drafts' pages (from the one that holds position ctx on) are not the request's own
    s["own_tables"] = s["tables"].clone()
    first = [x // c["bs"] for x in ctx]
    last = [-(-k // c["bs"]) for k in lens]
    fresh = torch.cat([torch.arange(f, k) + b * s["tables"].shape[1] for b, (f, k) in enumerate(zip(first, last))])
    s["own_tables"].view(-1)[fresh.to(DEV)] = blocks + torch.randperm(len(fresh), generator=g, device=DEV).to(torch.int32)
    blocks += len(fresh)
    s["ck"], s["cv"] = (normal(c["layers"], t, blocks, c["bs"], kv_per, HD) for _ in range(2))
    s["lk"], s["lv"] = list(s["ck"].unbind(0)), list(s["cv"].unbind(0))
    m = _accepted(c)
    acc = torch.full((c["reqs"], c["n"]), -1, dtype=torch.int32, device=DEV)
    for b in range(c["reqs"]):
        acc[b, :m[b]] = torch.randperm(n[b], generator=g, device=DEV)[:m[b]].sort().values.to(torch.int32)
    s["acc"] = acc
    s["new_lens"] = torch.empty(c["reqs"], dtype=torch.int32, device=DEV)
    s["ws"] = torch.zeros(16, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------- one pass
def run(s):
    op = s["c"]["op"]
    if op == "rope":
        if own:
            s["blk"].qk_norm_rope(s["qkv"], s["pos"], s["rope"], out=s["out"], slot_mapping=s["slots"],
                                  cache_k=s["ck"], cache_v=s["cv"], ws=s["ws"])
            out = s["out"]
        else:
            out = _rope_plain(s)
        return {"qkv": out, "cache_k": s["ck"], "cache_v": s["cv"]} if s["c"]["write"] else {"qkv": out}
    if op == "tree":
        if own:
            import tensor_linear_layers_gb300 as tl
            tl.tree_mask(s["parents"], s["qsl"], s["lens"], s["n"], out=(s["mask"], s["pos"]), ws=s["ws"])
            s["blk"].tree_attention(s["qkv"], s["qsl"], s["lens"], s["tables"], s["mask"], s["ck"], s["cv"], s["n"],
                                    s["max_len"], out=s["out"], ws=s["ws"])
            return {"out": s["out"], "mask": s["mask"], "pos": s["pos"]}
        return _tree_plain(s)
    if op == "fork":
        if own:
            s["blk"].kv_cache_copy_blocks(s["pairs"], s["lk"], s["lv"], ws=s["ws"])
        else:
            src, dst = s["pairs"].long().unbind(1)
            s["ck"][:, :, dst] = s["ck"][:, :, src]
            s["cv"][:, :, dst] = s["cv"][:, :, src]
        return {"cache_k": s["ck"], "cache_v": s["cv"]}
    if own:
        s["blk"].kv_cache_compact(s["qsl"], s["lens"], s["acc"], s["tables"], s["own_tables"], s["lk"], s["lv"],
                                  out=s["new_lens"], ws=s["ws"])
        return {"cache_k": s["ck"], "cache_v": s["cv"], "lens": s["new_lens"]}
    return _compact_plain(s)


def _rope_plain(s):
    c = s["c"]
    q_per, kv_per, _ = _shape(c)
    t, T, rd = c["t"], c["T"], c["rd"]
    x = s["qkv"].view(t, T, q_per + 2 * kv_per, HD)
    heads = x[:, :, :q_per + kv_per].float()
    if c["norm"]:
        gamma = torch.cat([s["gq"].expand(q_per, HD), s["gk"].expand(kv_per, HD)]).float()
        heads = heads * torch.rsqrt(heads.square().mean(-1, keepdim=True) + EPS) * gamma
    pos = s["pos"].long()
    cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
    if c["half"]:
        a, b = heads[..., :rd // 2], heads[..., rd // 2:rd]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = heads[..., 0:rd:2], heads[..., 1:rd:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    turned = torch.cat([turned, heads[..., rd:]], -1).to(torch.bfloat16)
    out = torch.cat([turned, x[:, :, q_per + kv_per:]], 2)
    if c["write"]:
        slots = s["slots"].long()
        s["ck"].view(t, -1, kv_per, HD)[:, slots] = out[:, :, q_per:q_per + kv_per]
        s["cv"].view(t, -1, kv_per, HD)[:, slots] = out[:, :, q_per + kv_per:]
    return out.view(t, T, -1)


def _tree_plain(s):
    c = s["c"]
    q_per, kv_per, _ = _shape(c)
    t, n, gq = c["t"], s["n"], q_per // kv_per
    qsl, lens = s["qsl"].long(), s["lens"].long()
    num = qsl[1:] - qsl[:-1]
    ctx = lens - num
    # drafted tokens padded to [request][n]; a padded one is its own root
    i = torch.arange(n, device=DEV)
    real = i < num[:, None]
    row = (qsl[:-1, None] + i).clamp(max=s["qkv"].shape[1] - 1)
    parent = torch.where(real, s["parents"].long()[row], -1)
    # ancestors: the closure of "is the parent of", by squaring
    sees = ((parent[:, :, None] == i) | (i[:, None] == i)).float()
    for _ in range(max(1, (n - 1).bit_length())):
        sees = ((sees @ sees) > 0).float()
    sees = sees > 0
    depth = sees.sum(-1) - 1
    bits = torch.zeros(*sees.shape[:2], s["words"] * 32, dtype=torch.int64, device=DEV)
    bits[:, :, :n] = sees.long()
    words = (bits.view(*sees.shape[:2], s["words"], 32) << torch.arange(32, device=DEV)).sum(-1)
    words = torch.where(words >= 2 ** 31, words - 2 ** 32, words)
    # every request's keys and values, padded to the longest
    key = torch.arange(s["max_len"], device=DEV)
    live = key < lens[:, None]
    page = s["tables"].long()[:, (key // c["bs"]).clamp(max=s["tables"].shape[1] - 1)]
    slot = torch.where(live, page * c["bs"] + key % c["bs"], 0)
    k = s["ck"].view(t, -1, kv_per, HD)[:, slot].float().permute(0, 1, 3, 4, 2)     # t, b, kv, hd, key
    v = s["cv"].view(t, -1, kv_per, HD)[:, slot].float().permute(0, 1, 3, 2, 4)     # t, b, kv, key, hd
    q = s["qkv"][:, row, :q_per * HD].float().view(t, c["reqs"], n, kv_per, gq, HD).permute(0, 1, 3, 4, 2, 5)
    score = (q.reshape(t, c["reqs"], kv_per, gq * n, HD) @ k).view(t, c["reqs"], kv_per, gq, n, -1) / math.sqrt(HD)
    draft = (key - ctx[:, None])                                                    # b, key
    pick = torch.gather(sees, 2, draft.clamp(0, n - 1)[:, None, :].expand(-1, n, -1))
    seen = live[:, None] & ((draft < 0)[:, None] | pick)                            # b, n, key
    score = score.masked_fill_(~seen[None, :, None, None], -math.inf)
    p = score.sub_(score.amax(-1, keepdim=True)).exp_()
    p = p.div_(p.sum(-1, keepdim=True))
    o = (p.view(t, c["reqs"], kv_per, gq * n, -1) @ v).view(t, c["reqs"], kv_per, gq, n, HD)
    o = o.permute(0, 1, 4, 2, 3, 5).reshape(t, c["reqs"], n, q_per * HD)
    return {"out": o[:, real].to(torch.bfloat16), "mask": words[real].to(torch.int32),
            "pos": (ctx[:, None] + depth)[real].to(torch.int32)}


def _compact_plain(s):
    c = s["c"]
    acc = s["acc"].long()
    ctx = (s["lens"] - s["qsl"][1:] + s["qsl"][:-1]).long()
    kept = acc >= 0
    old, new = ctx[:, None] + acc, ctx[:, None] + torch.arange(acc.shape[1], device=DEV)
    b = torch.arange(c["reqs"], device=DEV)[:, None].expand_as(acc)[kept]
    old, new = old[kept], new[kept]
    src = s["tables"].long()[b, old // c["bs"]] * c["bs"] + old % c["bs"]
    dst = s["own_tables"].long()[b, new // c["bs"]] * c["bs"] + new % c["bs"]
    for cache in (s["ck"], s["cv"]):
        flat = cache.view(c["layers"], c["t"], -1, cache.shape[-2], HD)
        flat[:, :, dst] = flat[:, :, src]
    return {"cache_k": s["ck"], "cache_v": s["cv"], "lens": (ctx + kept.sum(1)).to(torch.int32)}


# ---------------------------------------------------------------------------------------------- in 64 bits
def _exact_angles(c, pos):
    """cos and sin of every token's angles, from the frequencies' definition pair by pair."""
    rd, out = c["rd"], []
    for i in range(rd // 2):
        f = ROPE_BASE ** (-2.0 * i / rd)
        if c["scaling"] == "linear":
            f /= ROPE_FACTOR
        elif c["scaling"] == "ntk":
            f = (ROPE_BASE * ROPE_FACTOR ** (rd / (rd - 2.0))) ** (-2.0 * i / rd)
        elif c["scaling"] == "bands":
            wave = 2 * math.pi / f
            if wave > ROPE_ORIGINAL / LOW_FREQ:
                f /= ROPE_FACTOR
            elif wave >= ROPE_ORIGINAL / HIGH_FREQ:
                mix = (ROPE_ORIGINAL / wave - LOW_FREQ) / (HIGH_FREQ - LOW_FREQ)
                f = (1 - mix) * f / ROPE_FACTOR + mix * f
        elif c["scaling"] == "yarn":
            def pair_of(turns):
                return rd * math.log(ROPE_ORIGINAL / (2 * math.pi * turns)) / (2 * math.log(ROPE_BASE))
            lo, hi = max(math.floor(pair_of(BETA_FAST)), 0), min(math.ceil(pair_of(BETA_SLOW)), rd - 1)
            ramp = min(1.0, max(0.0, (i - lo) / (hi - lo if hi > lo else 0.001)))
            f = f * (1 - ramp) + f / ROPE_FACTOR * ramp
        out.append(f)
    angle = pos.double()[:, None] * torch.tensor(out, dtype=torch.float64, device=DEV)
    m = _yarn_mscale() if c["scaling"] == "yarn" else 1.0
    return angle.cos() * m, angle.sin() * m


def exact(c, seed):
    s = prepare(c, seed)
    q_per, kv_per, _ = _shape(c)
    t = c["t"]
    if c["op"] == "rope":
        T, rd = c["T"], c["rd"]
        x = s["qkv"].double().view(t, T, -1, HD)
        out = x.clone()
        cos, sin = _exact_angles(c, s["pos"])
        for h in range(q_per + kv_per):
            y = x[:, :, h]
            if c["norm"]:
                y = y / (y.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * (s["gq"] if h < q_per else s["gk"]).double()
            at = torch.arange(rd // 2, device=DEV)
            a, b = (at, at + rd // 2) if c["half"] else (2 * at, 2 * at + 1)
            out[:, :, h] = y
            out[:, :, h, a] = y[..., a] * cos - y[..., b] * sin
            out[:, :, h, b] = y[..., b] * cos + y[..., a] * sin
        r = {"qkv": out.reshape(t, T, -1)}
        if c["write"]:
            slots = s["slots"].long()
            for name, cache, at in (("cache_k", s["ck"], q_per), ("cache_v", s["cv"], q_per + kv_per)):
                full = cache.double()
                full.view(t, -1, kv_per, HD)[:, slots] = out[:, :, at:at + kv_per]
                r[name] = full
        return r
    if c["op"] == "fork":
        ck, cv = s["ck"].clone(), s["cv"].clone()
        for a, b in s["pairs"].tolist():
            ck[:, :, b], cv[:, :, b] = s["ck"][:, :, a], s["cv"][:, :, a]
        return {"cache_k": ck, "cache_v": cv}
    ctx, n = _tree_sizes(c)
    start = s["qsl"].tolist()
    if c["op"] == "tree":
        out = torch.zeros(t, sum(n), q_per * HD, dtype=torch.float64, device=DEV)
        parents = s["parents"].tolist()
        mask, pos = [], []
        for b in range(c["reqs"]):
            L = ctx[b] + n[b]
            see = torch.ones(n[b], L, dtype=torch.bool)
            see[:, ctx[b]:] = False
            for i in range(n[b]):
                word, at, depth = [0] * s["words"], i, -1
                while at >= 0:
                    see[i, ctx[b] + at] = True
                    word[at // 32] |= 1 << (at % 32)
                    at, depth = parents[start[b] + at], depth + 1
                mask.append([x - 2 ** 32 if x >= 2 ** 31 else x for x in word])
                pos.append(ctx[b] + depth)
            see = see.to(DEV)
            where = torch.arange(L, device=DEV)
            slot = s["tables"][b, where // c["bs"]].long() * c["bs"] + where % c["bs"]
            for r in range(t):
                k = s["ck"][r].view(-1, kv_per, HD)[slot].double()
                v = s["cv"][r].view(-1, kv_per, HD)[slot].double()
                for h in range(q_per):
                    q = s["qkv"][r, start[b]:start[b + 1], h * HD:(h + 1) * HD].double()
                    kv = h // (q_per // kv_per)
                    e = torch.where(see, q @ k[:, kv].T / HD ** 0.5, -math.inf)
                    out[r, start[b]:start[b + 1], h * HD:(h + 1) * HD] = torch.softmax(e, -1) @ v[:, kv]
        return {"out": out, "mask": torch.tensor(mask, dtype=torch.int32), "pos": torch.tensor(pos, dtype=torch.int32)}
    acc, src, dst, bs = s["acc"].tolist(), s["tables"].tolist(), s["own_tables"].tolist(), c["bs"]
    ck, cv, new = s["ck"].clone(), s["cv"].clone(), []
    for b in range(c["reqs"]):
        kept = [a for a in acc[b] if a >= 0]
        for j, a in enumerate(kept):
            x, y = ctx[b] + a, ctx[b] + j
            for to, of in ((ck, s["ck"]), (cv, s["cv"])):
                to[:, :, dst[b][y // bs], y % bs] = of[:, :, src[b][x // bs], x % bs]
        new.append(ctx[b] + len(kept))
    return {"cache_k": ck, "cache_v": cv, "lens": torch.tensor(new, dtype=torch.int32)}
