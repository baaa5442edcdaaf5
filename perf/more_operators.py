"""Cases that measure a paged KV cache held in 8 bits and the attention that reads paged caches by chunks of new tokens.

Three operators, each in its plain form (elementary torch operations in 32 bits) and as the framework's call:

* ``write``   k and v of new tokens quantised into their cache slots: e4m3 codes, a power-of-two scale per head of a token
* ``read``    the values of cached tokens, given by their slots, back in bf16
* ``attend``  every request's new tokens (one, or a chunk) over its paged cache, causal, with an optional sliding
              window and a few first tokens that stay visible; the cache in bf16 or in 8 bits

Layouts are the framework's: qkv [t][T][q heads | k heads | v heads of the shard][128] bf16; caches
[t][blocks][block_size][kv heads of the shard][128], bf16 or e4m3 with one scale byte per head: 127 + e for 2^e.
"""
import math

import torch

own = False

HD = 128
DEV = "cuda"
E_LO, E_HI = -100, 118     # exponents of a scale
F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the new tokens of a decode batch of 32 requests: latency
        {"name": "write_decode", "op": "write", "T": 32, "nq": 32, "nkv": 8, "t": 4, "bs": 16},
        # a prefill of 8192 tokens
        {"name": "write_prefill", "op": "write", "T": 8192, "nq": 32, "nkv": 8, "t": 4, "bs": 16},
        # one request's prompt, looked at again
        {"name": "read_prompt", "op": "read", "n": 1021, "nq": 28, "nkv": 4, "t": 4, "bs": 24},
        # long prefixes handed to a path that takes bf16
        {"name": "read_long", "op": "read", "n": 65536, "nq": 32, "nkv": 8, "t": 4, "bs": 16},
        # one user of a windowed model, the next token: latency
        {"name": "decode_single", "op": "attend", "reqs": 1, "n": 1, "ctx_lo": 4001, "ctx_hi": 4001, "nq": 32, "nkv": 8,
         "t": 4, "bs": 16, "window": 1024, "sinks": 4, "q8": False},
        # a decode batch of 32 requests on the 8-bit cache
        {"name": "decode_batch", "op": "attend", "reqs": 32, "n": 1, "ctx_lo": 255, "ctx_hi": 4095, "nq": 32, "nkv": 8,
         "t": 4, "bs": 16, "window": 0, "sinks": 0, "q8": True},
        # a decode batch of a windowed model, long contexts of which it reads 4096 tokens and the first 4
        {"name": "decode_window", "op": "attend", "reqs": 48, "n": 1, "ctx_lo": 1000, "ctx_hi": 16000, "nq": 28,
         "nkv": 4, "t": 4, "bs": 32, "window": 4096, "sinks": 4, "q8": False},
        # four long documents on the 8-bit cache, 64 q heads
        {"name": "decode_long", "op": "attend", "reqs": 4, "n": 1, "ctx_lo": 130001, "ctx_hi": 131040, "nq": 64,
         "nkv": 8, "t": 8, "bs": 64, "window": 0, "sinks": 0, "q8": True},
        # a prompt of 4096 tokens, nothing cached before
        {"name": "prompt", "op": "attend", "reqs": 1, "n": 4096, "ctx_lo": 0, "ctx_hi": 0, "nq": 32, "nkv": 8, "t": 4,
         "bs": 16, "window": 0, "sinks": 0, "q8": False},
        # the last 2048 tokens of a long prompt, the rest on the 8-bit cache
        {"name": "chunk_long", "op": "attend", "reqs": 1, "n": 2048, "ctx_lo": 30001, "ctx_hi": 30001, "nq": 32,
         "nkv": 8, "t": 4, "bs": 16, "window": 0, "sinks": 0, "q8": True},
        # a step that mixes decoding requests with chunks of prompts, windowed, 8-bit, 7 q heads per kv head
        {"name": "mixed_window", "op": "attend", "reqs": 16, "n": 509, "ctx_lo": 0, "ctx_hi": 7000, "nq": 28, "nkv": 4,
         "t": 4, "bs": 32, "window": 1024, "sinks": 16, "q8": True},
    ]


HEADS = ((32, 8), (28, 4), (64, 8), (8, 2), (4, 4))


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("write", "read", "attend", "attend", "attend", "attend"))
    nq, nkv = rng.choice(HEADS)
    t = rng.choice([t for t in (1, 2, 4, 8) if nq % t == 0 and (nkv % t == 0 or t % nkv == 0)])
    c = {"op": op, "nq": nq, "nkv": nkv, "t": t, "bs": rng.choice((1, 8, 16, 24, 32, 64, 128))}
    if op == "write":
        return {**c, "T": _log(rng, 1, 8192)}
    if op == "read":
        return {**c, "n": _log(rng, 1, 65536)}
    reqs = _log(rng, 1, 64)
    n = 1 if rng.random() < 0.4 else _log(rng, 2, 4096)
    kv = max(nkv, t)
    # the scores, the cached keys and the new tokens of all requests stay within the largest listed cases'
    while reqs > 1 and reqs * n * nq > 4096 * 32:
        reqs -= 1
    most = min(2048 * 32 * 32000 // (reqs * n * nq), 4 * 130000 * 8 // (reqs * kv), 130000) - n
    hi = _log(rng, 16, max(17, most))
    window = rng.choice((0, 0, 1, _log(rng, 2, 8192), _log(rng, 16, 8192)))
    return {**c, "reqs": reqs, "n": n, "ctx_lo": rng.randint(0, hi), "ctx_hi": hi, "window": window,
            "sinks": rng.choice((0, 1, 4, rng.randint(1, 200))) if window else 0, "q8": rng.random() < 0.5}


# ---------------------------------------------------------------------------------------------- shapes
def _shape(c):
    q_per = c["nq"] // c["t"]
    kv_per = 1 if c["t"] >= c["nkv"] else c["nkv"] // c["t"]
    return q_per, kv_per, (q_per + 2 * kv_per) * HD


def _spread(n, lo, hi):
    """n whole numbers of [lo, hi], spread evenly in an irregular order (the case alone fixes them)."""
    return [lo + int((hi - lo + 1) * ((0.381966 + 0.618034 * i) % 1.0)) for i in range(n)]


def _sizes(c):
    """Cached tokens and new tokens of each request: chunks of n, or for several requests a mix of single tokens and chunks."""
    n = [c["n"]] * c["reqs"]
    if c["reqs"] > 2:
        n = [1 if i % 2 else k for i, k in enumerate(_spread(c["reqs"], max(1, c["n"] // 4), c["n"]))]
    return _spread(c["reqs"], c["ctx_lo"], c["ctx_hi"]), n


def work(c):
    q_per, kv_per, _ = _shape(c)
    t = c["t"]
    if c["op"] != "attend":
        n = c["T"] if c["op"] == "write" else c["n"]
        return {"bytes": n * (t * 2 * kv_per * (HD * 3 + 1) + 4), "flops": 0}
    keys = pairs = 0
    W, S = c["window"], c["sinks"]
    ctx, num = _sizes(c)
    for x, n in zip(ctx, num):
        L = x + n
        keys += L if not W else L - max(0, x - W + 1 - S)
        for p in range(x, L):
            pairs += p + 1 if not W else p + 1 - max(0, p - W + 1 - S)
    T = sum(num)
    per_key = HD + 1 if c["q8"] else 2 * HD
    b = keys * t * kv_per * 2 * per_key + 2 * T * t * q_per * HD * 2 + sum(-(-(x + n) // c["bs"]) for x, n in zip(ctx, num)) * 4
    return {"bytes": b, "flops": 4.0 * HD * c["nq"] * pairs}


# ---------------------------------------------------------------------------------------------- inputs
def _handle(c):
    """The framework's attention handle of these head counts (its projections are not used here)."""
    import tensor_linear_layers_gb300 as tl
    cfg = tl.make_config(tl.TP_BLOCK_ATTN_PROJ, c["t"], 256, n_q_heads=c["nq"], n_kv_heads=c["nkv"], head_dim=HD)
    z = torch.zeros(c["nq"] * HD * 256, dtype=torch.bfloat16, device=DEV)
    kv = z[:c["nkv"] * HD * 256].view(-1, 256)
    return tl.TPLinear(cfg, [z.view(-1, 256), kv, kv, z.view(256, -1)])


def _pow2(e):
    """2^e in 32 bits for whole e in [-126, 127]."""
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _quantised(x):
    """Codes and scale bytes of head rows [..., 128]: every product here is by a power of two, so 32 bits hold it exactly."""
    a = x.float()
    top = a.abs().amax(-1)
    m, e = torch.frexp(top)                                    # top = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(top > 0, e - 9 + (m > 0.875).to(e.dtype), E_LO).clamp(E_LO, E_HI)
    y = (a * _pow2(-e)[..., None]).clamp(-448, 448)
    return y.to(F8), (e + 127).to(torch.uint8)


def _values(codes, scales):
    """What codes and scale bytes stand for, in 32 bits (exact)."""
    return codes.float() * _pow2(scales.to(torch.int32) - 127)[..., None]


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    q_per, kv_per, w = _shape(c)
    t, bs = c["t"], c["bs"]
    s = {"c": c}

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)

    def uneven(x):
        # keys have a few strong channels, and tokens of different strength
        x *= torch.exp(0.6 * normal(HD))
        return x.mul_(torch.exp(0.4 * normal(*x.shape[:-1], 1)))

    if own:
        s["blk"] = _handle(c)
    s["ws"] = torch.zeros(16, dtype=torch.uint8, device=DEV)
    if c["op"] == "write":
        T = c["T"]
        s["qkv"] = uneven(normal(t, T, w // HD, HD)).view(t, T, w)
        blocks = -(-T // bs) + 4
        s["slots"] = torch.randperm(blocks * bs, generator=g, device=DEV)[:T].to(torch.int32)
        s["cache"] = [torch.zeros(t, blocks, bs, kv_per, HD, dtype=F8, device=DEV) for _ in range(2)]
        s["scale"] = [torch.full((t, blocks, bs, kv_per), 127, dtype=torch.uint8, device=DEV) for _ in range(2)]
        return s
    if c["op"] == "read":
        blocks = -(-c["n"] // bs) + 4
        at = torch.arange(-(-c["n"] // bs) * bs, device=DEV)
        perm = torch.randperm(blocks, generator=g, device=DEV)
        s["slots"] = (perm[at // bs] * bs + at % bs)[:c["n"]].to(torch.int32).contiguous()
        pairs = [_quantised(uneven(normal(t, blocks, bs, kv_per, HD))) for _ in range(2)]
        s["cache"], s["scale"] = [p[0] for p in pairs], [p[1] for p in pairs]
        s["out"] = [torch.empty(t, c["n"], kv_per, HD, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        return s
    ctx, n = _sizes(c)
    lens = [x + k for x, k in zip(ctx, n)]
    s["n"], s["max_len"] = max(n), max(lens)
    s["qsl"] = torch.tensor([sum(n[:b]) for b in range(len(n) + 1)], dtype=torch.int32, device=DEV)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    # scattered pages
    need = [-(-k // bs) for k in lens]
    blocks = sum(need) + 3
    perm = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor([sum(need[:b]) for b in range(len(need))], device=DEV)
    s["tables"] = perm[(first[:, None] + torch.arange(max(need), device=DEV)).clamp(max=blocks - 1)].contiguous()
    s["qkv"] = normal(t, sum(n), w)
    s["cache"] = [uneven(normal(t, blocks, bs, kv_per, HD)) for _ in range(2)]
    s["scale"] = [None, None]
    if c["q8"]:
        pairs = [_quantised(x) for x in s["cache"]]
        s["cache"], s["scale"] = [p[0] for p in pairs], [p[1] for p in pairs]
    s["out"] = torch.empty(t, sum(n), q_per * HD, dtype=torch.bfloat16, device=DEV)
    if own:
        size = s["blk"].chunk_attention_workspace_size(c["reqs"], s["n"], s["max_len"])
        s["ws"] = torch.zeros(size, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------- one pass
def run(s):
    op = s["c"]["op"]
    if op == "write":
        (ck, cv), (sk, sv) = s["cache"], s["scale"]
        if own:
            s["blk"].kv_quant_write(s["qkv"], s["slots"], ck, cv, sk, sv, ws=s["ws"])
        else:
            _write_plain(s)
        return {"codes_k": ck, "codes_v": cv, "scales_k": sk, "scales_v": sv}
    if op == "read":
        if own:
            s["blk"].kv_quant_read(s["slots"], *s["cache"], *s["scale"], out=s["out"], ws=s["ws"])
            return s["out"]
        return _read_plain(s)
    if own:
        s["blk"].chunk_attention(s["qkv"], s["qsl"], s["lens"], s["tables"], *s["cache"], s["n"], s["max_len"],
                                 window=s["c"]["window"], sinks=s["c"]["sinks"], scales_k=s["scale"][0],
                                 scales_v=s["scale"][1], out=s["out"], ws=s["ws"])
        return s["out"]
    return _attend_plain(s)


def _write_plain(s):
    c = s["c"]
    q_per, kv_per, _ = _shape(c)
    heads = s["qkv"].view(c["t"], c["T"], -1, HD)[:, :, q_per:]
    codes, scales = _quantised(heads)
    slots = s["slots"].long()
    bits = codes.view(torch.uint8)
    (ck, cv), (sk, sv) = s["cache"], s["scale"]
    ck.view(torch.uint8).view(c["t"], -1, kv_per, HD)[:, slots] = bits[:, :, :kv_per]
    cv.view(torch.uint8).view(c["t"], -1, kv_per, HD)[:, slots] = bits[:, :, kv_per:]
    sk.view(c["t"], -1, kv_per)[:, slots] = scales[:, :, :kv_per]
    sv.view(c["t"], -1, kv_per)[:, slots] = scales[:, :, kv_per:]


def _read_plain(s):
    c = s["c"]
    kv_per = _shape(c)[1]
    return [_picked(x, e, c["t"], kv_per, s["slots"].long()).to(torch.bfloat16) for x, e in zip(s["cache"], s["scale"])]


def _picked(cache, scale, t, kv_per, slots):
    """The cached heads at these slots, in 32 bits."""
    if scale is None:
        return cache.view(t, -1, kv_per, HD)[:, slots].float()
    codes = cache.view(torch.uint8).view(t, -1, kv_per, HD)[:, slots].view(F8)
    return _values(codes, scale.view(t, -1, kv_per)[:, slots])


def _attend_plain(s):
    c = s["c"]
    q_per, kv_per, _ = _shape(c)
    t, n, gq, bs = c["t"], s["n"], q_per // kv_per, c["bs"]
    qsl, lens = s["qsl"].long(), s["lens"].long()
    num = qsl[1:] - qsl[:-1]
    ctx = lens - num
    i = torch.arange(n, device=DEV)
    real = i < num[:, None]
    row = (qsl[:-1, None] + i).clamp(max=s["qkv"].shape[1] - 1)
    # every request's keys and values, padded to the longest
    key = torch.arange(s["max_len"], device=DEV)
    live = key < lens[:, None]
    page = s["tables"].long()[:, (key // bs).clamp(max=s["tables"].shape[1] - 1)]
    slot = torch.where(live, page * bs + key % bs, 0)
    k = _picked(s["cache"][0], s["scale"][0], t, kv_per, slot).permute(0, 1, 3, 4, 2)     # t, b, kv, hd, key
    v = _picked(s["cache"][1], s["scale"][1], t, kv_per, slot).permute(0, 1, 3, 2, 4)     # t, b, kv, key, hd
    q = s["qkv"][:, row, :q_per * HD].float().view(t, c["reqs"], n, kv_per, gq, HD).permute(0, 1, 3, 4, 2, 5)
    score = (q.reshape(t, c["reqs"], kv_per, gq * n, HD) @ k).div_(math.sqrt(HD)).view(t, c["reqs"], kv_per, gq, n, -1)
    pos = (ctx[:, None] + i)[:, :, None]                                                  # b, n, 1
    seen = live[:, None] & (key <= pos)
    if c["window"]:
        seen &= (key > pos - c["window"]) | (key < c["sinks"])
    seen |= ~real[:, :, None]                # a padded row takes everything and is dropped
    score.masked_fill_(~seen[None, :, None, None], -math.inf)
    p = score.sub_(score.amax(-1, keepdim=True)).exp_()
    p = p.div_(p.sum(-1, keepdim=True))
    o = (p.view(t, c["reqs"], kv_per, gq * n, -1) @ v).view(t, c["reqs"], kv_per, gq, n, HD)
    o = o.permute(0, 1, 4, 2, 3, 5).reshape(t, c["reqs"], n, q_per * HD)
    return o[:, real].to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------- in 64 bits
def _power(e):
    """2^e in 64 bits for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_codes(x):
    """Values of the nearest codes and the scale exponents of head rows, from the formats' definition."""
    a = x.double()
    top = a.abs().amax(-1)
    e = torch.ceil(torch.log2(top / 448.0)).clamp(E_LO, E_HI)
    # (a logarithm may be off by one at a power of two)
    e = torch.where((top <= 448.0 * _power(e - 1)) & (e > E_LO), e - 1, e)
    e = torch.where((top > 448.0 * _power(e)) & (e < E_HI), e + 1, e)
    y = (a / _power(e)[..., None]).clamp(-448, 448)
    low = y.abs().clamp(min=2.0 ** -6)
    bits = torch.frexp(low)[1] - 1                             # 2^bits <= low < 2^(bits + 1)
    step = _power(bits - 3)
    return torch.round(y / step) * step, e


def exact(c, seed):
    s = prepare(c, seed)
    q_per, kv_per, _ = _shape(c)
    t, bs = c["t"], c["bs"]
    if c["op"] == "write":
        x = s["qkv"].view(t, c["T"], -1, HD)
        r = {}
        for name, at, cache, scale in (("k", q_per, *[z[0] for z in (s["cache"], s["scale"])]),
                                       ("v", q_per + kv_per, *[z[1] for z in (s["cache"], s["scale"])])):
            y, e = _exact_codes(x[:, :, at:at + kv_per])
            full, exps = cache.float().double(), scale.long()
            full.view(t, -1, kv_per, HD)[:, s["slots"].long()] = y
            exps.view(t, -1, kv_per)[:, s["slots"].long()] = e.long() + 127
            r["codes_" + name], r["scales_" + name] = full, exps
        return r
    if c["op"] == "read":
        at = s["slots"].long()
        return [x.float().double().view(t, -1, kv_per, HD)[:, at] * _power(e.long() - 127).view(t, -1, kv_per, 1)[:, at]
                for x, e in zip(s["cache"], s["scale"])]
    ctx, n = _sizes(c)
    start = s["qsl"].tolist()
    out = torch.zeros(t, sum(n), q_per * HD, dtype=torch.float64, device=DEV)
    for b in range(c["reqs"]):
        L = ctx[b] + n[b]
        where = torch.arange(L, device=DEV)
        slot = s["tables"][b, where // bs].long() * bs + where % bs
        # rows of 512 tokens at a time: position minus key, by hand
        for r in range(t):
            kv = []
            for x, e in zip(s["cache"], s["scale"]):
                if e is None:
                    kv.append(x[r].view(-1, kv_per, HD)[slot].double())
                else:
                    raw = x[r].view(torch.uint8).view(-1, kv_per, HD)[slot].view(F8).float().double()
                    kv.append(raw * _power(e[r].view(-1, kv_per, 1)[slot].long() - 127))
            for i0 in range(0, n[b], 512):
                i1 = min(n[b], i0 + 512)
                dist = torch.arange(ctx[b] + i0, ctx[b] + i1, device=DEV)[:, None] - where
                hide = dist < 0
                if c["window"] > 0:
                    hide |= (dist >= c["window"]) & (where >= c["sinks"])
                for h in range(q_per):
                    g = h // (q_per // kv_per)
                    q = s["qkv"][r, start[b] + i0:start[b] + i1, h * HD:(h + 1) * HD].double()
                    e = (q @ kv[0][:, g].T / HD ** 0.5).masked_fill_(hide, -math.inf)
                    out[r, start[b] + i0:start[b] + i1, h * HD:(h + 1) * HD] = torch.softmax(e, -1) @ kv[1][:, g]
    return out
