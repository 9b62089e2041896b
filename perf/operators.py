"""The decode-step operators around the verify step, at the sizes they are measured at.

Four operators of one decode step of a model that drafts and verifies tokens: the drafted tokens' keys and values
go into a paged cache (``kv_append``), the tokens attend over it (``paged_attention``), the verified branch's cache
entries move up behind the context (``kv_keep``), and the logits of every drafted position are shaped by the
request's penalties, biases and grammar before they are verified (``process_logits``).

``run`` computes them in elementary torch operations, or, where ``own`` is true, through this package's calls.
"""
from __future__ import annotations

import math

import torch

own = False

F8 = torch.float8_e4m3fn
F8_MAX = 448.0
ROPE_BASE = 10000.0


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # one stream decoding one token: all launch latency
        dict(name="attend one token", op="attend", B=1, T=1, Hq=8, Hkv=2, D=64, page=16, ctx_lo=515, ctx_hi=515,
             cache="bf16", chains=0, ragged=False, layout="slot"),
        # a small batch verifying chains of 5 drafts, contexts from empty to a few thousand tokens
        dict(name="attend chains", op="attend", B=8, T=6, Hq=32, Hkv=8, D=128, page=16, ctx_lo=0, ctx_hi=4001,
             cache="bf16", chains=0, ragged=True, layout="slot"),
        # a serving batch of 64 requests with 6 drafts each: the cache is read at memory speed
        dict(name="attend batch", op="attend", B=64, T=7, Hq=32, Hkv=8, D=128, page=32, ctx_lo=1000, ctx_hi=16000,
             cache="bf16", chains=0, ragged=True, layout="head"),
        # two long documents: few rows, so the work is the split over the cache's length
        dict(name="attend long", op="attend", B=2, T=5, Hq=32, Hkv=4, D=128, page=64, ctx_lo=100003, ctx_hi=131071,
             cache="bf16", chains=0, ragged=False, layout="head"),
        # four draft chains of four tokens as a tree over an 8-bit cache
        dict(name="attend tree 8-bit", op="attend", B=32, T=17, Hq=32, Hkv=8, D=128, page=16, ctx_lo=500, ctx_hi=9000,
             cache="e4m3", chains=4, ragged=False, layout="head"),
        # the drafted tokens of a small batch
        dict(name="append drafts", op="append", B=8, T=6, Hq=32, Hkv=8, D=128, page=16, ctx_lo=0, ctx_hi=4001,
             cache="bf16", chains=0, ragged=True, layout="slot", interleaved=False, rot=128),
        # a chunk of prompts going into an 8-bit cache
        dict(name="append prompts 8-bit", op="append", B=4, T=2047, Hq=32, Hkv=8, D=128, page=32, ctx_lo=1, ctx_hi=130,
             cache="e4m3", chains=0, ragged=True, layout="head", interleaved=True, rot=64),
        # one layer of one small batch
        dict(name="keep one layer", op="keep", L=1, B=4, T=9, Hkv=8, D=128, page=16, ctx_lo=17, ctx_hi=300,
             cache="bf16", chains=2, layout="slot"),
        # every layer of a serving batch at once
        dict(name="keep all layers", op="keep", L=32, B=64, T=17, Hkv=8, D=128, page=16, ctx_lo=30, ctx_hi=200,
             cache="bf16", chains=4, layout="head"),
        # the smallest verify workload
        dict(name="logits one request", op="logits", B=1, T=5, V=1000, dtype="f32", L=300, mask=True, bias=8,
             penalties=True, ragged=False),
        # 64 requests of 6 drafts, half of them under a tight grammar
        dict(name="logits grammar", op="logits", B=64, T=7, V=128256, dtype="bf16", L=2048, mask=True, bias=300,
             penalties=True, ragged=False),
        # the largest vocabulary in 32 bits, ragged drafts, long histories, no grammar
        dict(name="logits ragged", op="logits", B=256, T=9, V=152064, dtype="f32", L=4000, mask=False, bias=20,
             penalties=True, ragged=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "append", "keep", "logits", "logits"))
    if op == "logits":
        dtype = rng.choice(("f32", "bf16"))
        V = _log_int(rng, 300, 152064)
        if rng.random() < 0.7:
            V -= V % 8
        T = rng.randint(1, 17)
        most = 1.0e9 / (V * T * (8 if dtype == "f32" else 4))
        return dict(op=op, B=_log_int(rng, 1, max(1, min(512, int(most)))), T=T, V=V, dtype=dtype,
                    L=_log_int(rng, 1, 8000), mask=rng.random() < 0.5, bias=rng.choice((0, 1, 17, 300)),
                    penalties=rng.random() < 0.8, ragged=rng.random() < 0.5)
    c = dict(op=op, Hkv=rng.choice((1, 2, 4, 5, 8)), D=rng.choice((64, 128)), page=rng.choice((8, 16, 32, 64, 128, 256)),
             cache=rng.choice(("bf16", "e4m3")), layout=rng.choice(("slot", "head")))
    group = rng.choice((1, 2, 3, 4, 7, 8, 16))
    chains = 0
    T = rng.choice((1, 1, 2, 3, 4, 5, 6, 7, 8, 9, 13, 17))
    if op == "keep" or rng.random() < 0.25:
        chains = rng.randint(2, 4)
        T = 1 + chains * rng.randint(1, 12)
    slot_bytes = c["Hkv"] * c["D"] * 4
    if op == "keep":
        L = _log_int(rng, 1, 40)
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, max(1, min(2000, int(6e8 / (L * B * slot_bytes)))))
        return dict(c, L=L, B=B, T=T, chains=chains, ctx_lo=rng.randint(0, hi), ctx_hi=hi)
    if op == "append":
        if not chains and rng.random() < 0.4:
            T = _log_int(rng, 17, 4000)
        B = _log_int(rng, 1, max(1, min(256, int(3e8 / (T * (group + 2) * c["Hkv"] * c["D"] * 4)))))
        hi = _log_int(rng, 1, max(1, min(4000, int(5e8 / (B * slot_bytes)))))
        return dict(c, B=B, T=T, Hq=group * c["Hkv"], chains=chains, ctx_lo=rng.randint(0, hi), ctx_hi=hi,
                    ragged=rng.random() < 0.5, interleaved=rng.random() < 0.5, rot=rng.choice((0, 32, 64, c["D"])))
    most = min(6e8 / slot_bytes, 3e10 / (4 * T * group * c["Hkv"] * c["D"]))  # cache slots of all requests together
    hi = _log_int(rng, 1, max(1, min(131072, int(most))))
    B = _log_int(rng, 1, max(1, min(256, int(most / hi))))
    return dict(c, B=B, T=T, Hq=group * c["Hkv"], chains=chains, ctx_lo=rng.randint(0, hi), ctx_hi=hi,
                ragged=rng.random() < 0.5)


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def _spread(lo, hi, n):
    """n whole numbers evenly spread over [lo, hi] (the same for every seed; prepare() shuffles them)."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _tokens(case):
    """Valid new tokens of each request."""
    B, T = case["B"], case["T"]
    return _spread(min(3, T), T, B) if case.get("ragged") else [T] * B


def _tree(T, chains):
    """A root and `chains` chains behind it: each token's depth, and the bits of the new tokens it attends to."""
    K = (T - 1) // chains
    depth, bits = [0], [1]
    for n in range(chains):
        seen = 1
        for j in range(K):
            i = 1 + n * K + j
            seen |= 1 << i
            depth.append(j + 1)
            bits.append(seen - (1 << 64) if seen >= 1 << 63 else seen)
    return depth, bits


def _cache(case, layers, num_pages, g):
    """A pool of pages [layers, pages, page, heads, D] as views of the asked memory order."""
    dev, H, D, ps = "cuda", case["Hkv"], case["D"], case["page"]
    shape = (layers, num_pages, H, ps, D) if case["layout"] == "head" else (layers, num_pages, ps, H, D)
    pool = []
    for _ in range(2):
        x = torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(0.0, 1.0, generator=g)
        if case["cache"] == "e4m3":
            x = x.to(F8)
        pool.append(x.transpose(2, 3) if case["layout"] == "head" else x)
    return pool


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    B, T = case["B"], case["T"]
    i32 = dict(dtype=torch.int32, device=dev)
    order = torch.randperm(B, generator=g, device=dev)
    s = dict(case=case)
    s["t_per_row"] = torch.tensor(_tokens(case), **i32)[order] if case.get("ragged") else None
    if case["op"] == "logits":
        V, L = case["V"], case["L"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s["logits"] = torch.empty((B, T, V), dtype=dt, device=dev).normal_(0.0, 3.0, generator=g)
        s["out"] = torch.zeros_like(s["logits"])  # rows past a request's tokens stay as they are
        u = torch.rand((B, L + T - 1), generator=g, device=dev)
        ids = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1).to(torch.int32)  # frequent tokens repeat
        s["history"], s["draft"] = ids[:, :L].contiguous(), ids[:, L:].contiguous()
        s["history_len"] = torch.tensor(_spread(L // 2, L, B), **i32)[order]
        s["prompt_len"] = s["history_len"] // 3
        one = lambda lo, hi: torch.rand(B, generator=g, device=dev) * (hi - lo) + lo  # noqa: E731
        pen = case["penalties"]
        s["repetition"], s["presence"], s["frequency"] = (one(1.0, 1.4), one(0.0, 0.8), one(0.0, 0.4)) if pen else (None,) * 3
        n = min(case["bias"], V)
        s["bias_ids"] = s["bias"] = None
        if n:
            first = torch.randint(0, V, (B, 1), generator=g, device=dev)
            s["bias_ids"] = ((first + torch.arange(n, device=dev) * max(1, V // n)) % V).to(torch.int32)  # all different
            s["bias"] = torch.empty((B, n), device=dev).normal_(0.0, 2.0, generator=g)
        s["mask"] = None
        if case["mask"]:
            words = lambda: torch.randint(-2 ** 31, 2 ** 31, (B, T, (V + 31) // 32), generator=g, device=dev).to(torch.int32)  # noqa: E731
            a, b, c, d = words(), words(), words(), words()
            tight = (torch.arange(B, device=dev) % 2 == 0)[:, None, None]
            s["mask"] = torch.where(tight, a & b & c & d, a | b | c | d).contiguous()
        return s

    ctx = _spread(case["ctx_lo"], case["ctx_hi"], B)
    maxp = -(-(case["ctx_hi"] + T) // case["page"])
    num_pages = B * maxp + 3
    s["pages"] = torch.randperm(num_pages, generator=g, device=dev)[: B * maxp].to(torch.int32).view(B, maxp)
    s["ctx_len"] = torch.tensor(ctx, **i32)[B - 1 - order]
    layers = case.get("L", 1)
    k, v = _cache(case, layers, num_pages, g)
    H, D = case["Hkv"], case["D"]
    if case["op"] == "keep":
        s["k_cache"], s["v_cache"] = k, v
        K = (T - 1) // case["chains"]
        chain = torch.randint(0, case["chains"], (B, 1), generator=g, device=dev)
        s["path"] = torch.cat([torch.zeros_like(chain), 1 + chain * K + torch.arange(K, device=dev)], 1).to(torch.int32)
        s["n_keep"] = torch.tensor(_spread(1, K + 1, B), **i32)[order]  # the root and the accepted drafts
        return s
    s["k_cache"], s["v_cache"] = k[0], v[0]
    s["k_scale"] = s["v_scale"] = None
    if case["cache"] == "e4m3":
        s["k_scale"] = torch.rand(H, generator=g, device=dev) * 0.02 + 0.99
        s["v_scale"] = torch.rand(H, generator=g, device=dev) * 0.5 + 0.1
    normal = lambda h, sd: torch.empty((B, T, h, D), dtype=torch.bfloat16, device=dev).normal_(0.0, sd, generator=g)  # noqa: E731
    s["positions"] = s["mask"] = None
    if case["chains"]:
        depth, bits = _tree(T, case["chains"])
        s["mask"] = torch.tensor(bits, dtype=torch.int64, device=dev).expand(B, T).contiguous()
        s["positions"] = s["ctx_len"][:, None] + torch.tensor(depth, **i32)
    if case["op"] == "attend":
        s["q"] = normal(case["Hq"], 2.0)
        s["scale"] = 1.0 / math.sqrt(D)
        return s
    # one projection's output holds the heads of q, k and v side by side
    qkv = normal(case["Hq"] + 2 * H, 1.5)
    s["q"], s["k"], s["v"] = qkv[:, :, : case["Hq"]], qkv[:, :, case["Hq"]: case["Hq"] + H], qkv[:, :, case["Hq"] + H:]
    s["cos"] = s["sin"] = None
    if case["rot"]:
        n = case["ctx_hi"] + T
        freq = ROPE_BASE ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
        angle = torch.arange(n, device=dev, dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    s["out"] = torch.zeros((B, T, case["Hq"], D), dtype=torch.bfloat16, device=dev)
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        import speculative_decoding_rejection_verify_gb300 as sv
        if op == "attend":
            return sv.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["ctx_len"], s["t_per_row"],
                                      mask=s["mask"], scale=s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"])
        if op == "append":
            q = sv.kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["pages"], s["ctx_len"], s["cos"],
                             s["sin"], s["t_per_row"], positions=s["positions"], interleaved=s["case"]["interleaved"],
                             k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"])
            return [q, s["k_cache"], s["v_cache"]]
        if op == "keep":
            sv.kv_keep(s["k_cache"], s["v_cache"], s["pages"], s["ctx_len"], s["path"], s["n_keep"])
            return [s["k_cache"], s["v_cache"]]
        return sv.process_logits(s["logits"], history=s["history"], history_len=s["history_len"],
                                 prompt_len=s["prompt_len"], draft=s["draft"], t_per_row=s["t_per_row"],
                                 repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                                 bias_ids=s["bias_ids"], bias=s["bias"], mask=s["mask"], out=s["out"])
    return {"attend": _attend, "append": _append, "keep": _keep, "logits": _logits}[op](s)


def _count(s):
    """[B] valid new tokens."""
    t = s["t_per_row"]
    return t if t is not None else torch.full((s["case"]["B"],), s["case"]["T"], dtype=torch.int32, device="cuda")


def _gather(cache, pages, scale):
    """The cache of every request side by side, [B, slots, heads, D] in 32 bits."""
    raw = cache.view(torch.uint8) if cache.dtype == F8 else cache
    x = raw[pages.long()]
    x = (x.view(F8) if cache.dtype == F8 else x).flatten(1, 2).float()
    return x if scale is None else x * scale[:, None]


def _attend(s):
    q, tb, ctx = s["q"], _count(s), s["ctx_len"]
    B, T, Hq, D = q.shape
    H = s["k_cache"].shape[2]
    k, v = (_gather(s[n + "_cache"], s["pages"], s[n + "_scale"]) for n in "kv")
    S = k.shape[1]
    t = torch.arange(T, device=q.device)
    new = torch.arange(S, device=q.device) - ctx[:, None]  # [B, S]: which new token a slot holds, negative in the context
    if s["mask"] is None:
        sees = new[:, None] <= t[:, None]
    else:
        sees = (new[:, None] < 0) | ((s["mask"][:, :, None] >> new[:, None].clamp(0, 63)) & 1).bool()
    sees = sees & (new < tb[:, None])[:, None] & (t < tb[:, None])[:, :, None]
    v = torch.where((new < tb[:, None])[:, :, None, None], v, 0.0)
    rows = q.float().view(B, T, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, -1, D)
    z = torch.matmul(rows, k.permute(0, 2, 3, 1)).view(B, H, Hq // H, T, S) * s["scale"]
    z = z.masked_fill(~sees[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, H, -1, S), v.permute(0, 2, 1, 3)).view(B, H, Hq // H, T, D)
    o = torch.where(total > 0, o / total, 0.0)
    return o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(q.dtype)


def _rotate(x, cos, sin, interleaved):
    r = 2 * cos.shape[-1]
    cos, sin = cos[:, :, None], sin[:, :, None]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., : r // 2], x[..., r // 2: r])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _append(s):
    B, T = s["case"]["B"], s["case"]["T"]
    ctx, dev = s["ctx_len"], s["q"].device
    t = torch.arange(T, device=dev)
    slot = (ctx[:, None] + t).long()
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if s["cos"] is not None:
        at = slot if s["positions"] is None else s["positions"].long()
        cos, sin = s["cos"][at], s["sin"][at]
        q, k = (_rotate(x, cos, sin, s["case"]["interleaved"]) for x in (q, k))
    valid = t < _count(s)[:, None]
    s["out"].copy_(torch.where(valid[:, :, None, None], q, 0.0))
    page = s["case"]["page"]
    where = torch.gather(s["pages"].long(), 1, slot // page)[valid], (slot % page)[valid]
    for name, x in (("k", k), ("v", v)):
        cache, scale = s[name + "_cache"], s[name + "_scale"]
        x = x[valid]
        if cache.dtype == F8:
            x = (x / scale[:, None]).clamp(-F8_MAX, F8_MAX).to(F8).view(torch.uint8)
            cache.view(torch.uint8)[where] = x
        else:
            cache[where] = x.to(cache.dtype)
    return [s["out"], s["k_cache"], s["v_cache"]]


def _keep(s):
    page, path = s["case"]["page"], s["path"].long()
    i = torch.arange(path.shape[1], device=path.device)
    valid = i < s["n_keep"][:, None]
    place = lambda n: (torch.gather(s["pages"].long(), 1, n // page)[valid], (n % page)[valid])  # noqa: E731
    source, target = place(s["ctx_len"][:, None] + path), place(s["ctx_len"][:, None] + i)
    for name in ("k_cache", "v_cache"):
        cache = s[name].view(torch.uint8) if s[name].dtype == F8 else s[name]
        cache[:, target[0], target[1]] = cache[:, source[0], source[1]]
    return [s["k_cache"], s["v_cache"]]


def _logits(s):
    z, dev = s["logits"].float(), s["logits"].device
    B, T, V = z.shape
    n = torch.arange(s["history"].shape[1], device=dev)
    held = n < s["history_len"][:, None]
    prompt = held & (n < s["prompt_len"][:, None])
    ids = s["history"].long()
    count = torch.zeros((B, V), device=dev).scatter_add_(1, ids, (held & ~prompt).float())
    seen = torch.zeros((B, V), device=dev).scatter_add_(1, ids, prompt.float())
    step = torch.zeros((B, T, V), device=dev)
    step[torch.arange(B, device=dev)[:, None], torch.arange(1, T, device=dev), s["draft"].long()] = 1.0
    count = count[:, None] + step.cumsum(1)  # position t also holds the drafts before it
    if s["repetition"] is not None:
        r = s["repetition"][:, None, None]
        z = torch.where((count > 0) | (seen[:, None] > 0), torch.where(z > 0, z / r, z * r), z)
        z = z - s["frequency"][:, None, None] * count - s["presence"][:, None, None] * (count > 0).float()
    if s["bias"] is not None:
        z = z + torch.zeros((B, V), device=dev).scatter_add_(1, s["bias_ids"].long(), s["bias"])[:, None]
    if s["mask"] is not None:
        bits = (s["mask"][..., None] >> torch.arange(32, device=dev, dtype=torch.int32)) & 1
        z = z.masked_fill(bits.flatten(-2)[..., :V] == 0, -math.inf)
    valid = torch.arange(T, device=dev) < _count(s)[:, None]
    s["out"].copy_(torch.where(valid[:, :, None], z, s["out"].float()))
    return s["out"]


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# ------------------------------------------------------------------------------------------------
def work(case):
    B, op = case["B"], case["op"]
    if op == "logits":
        es, rows, V = (4 if case["dtype"] == "f32" else 2), sum(_tokens(case)), case["V"]
        b = rows * V * es * 2 + sum(_spread(case["L"] // 2, case["L"], B)) * 4 + B * case["bias"] * 8
        return {"bytes": b + (rows * ((V + 31) // 32) * 4 if case["mask"] else 0), "flops": rows * V}
    es = 2 if case["cache"] == "bf16" else 1
    slot = case["Hkv"] * case["D"]
    if op == "keep":
        K = (case["T"] - 1) // case["chains"]
        moved = sum(n - 1 for n in _spread(1, K + 1, B)) * (case["chains"] - 1) / case["chains"]  # the first chain stays
        return {"bytes": case["L"] * moved * slot * es * 2 * 2 + B * (K + 3) * 4, "flops": 0}
    tokens = sum(_tokens(case))
    q = tokens * case["Hq"] * case["D"] * 2
    if op == "append":
        table = tokens * case["rot"] * 4
        return {"bytes": 2 * q + tokens * slot * 2 * (2 + es) + table + 8 * B,
                "flops": 3 * tokens * (case["Hq"] + case["Hkv"]) * case["rot"]}
    pairs = [(c + t) for c, t in zip(_spread(case["ctx_lo"], case["ctx_hi"], B), _tokens(case)[::-1])]
    flops = sum(4 * n * t for n, t in zip(pairs, _tokens(case)[::-1])) * case["Hq"] * case["D"]
    return {"bytes": 2 * q + sum(pairs) * slot * 2 * es + sum(-(-n // case["page"]) for n in pairs) * 4, "flops": flops}


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _attend64, "append": _append64, "keep": _keep64, "logits": _logits64}[case["op"]](s)


def _slots64(s, name, b, slots):
    """Cache entries of request b in 64 bits, [slots, heads, D]."""
    page = s["case"]["page"]
    at = s["pages"][b].long()[slots // page] * page + slots % page
    cache = s[name + "_cache"]
    raw = cache.contiguous().view(torch.uint8).view(cache.shape[0] * page, cache.shape[2], -1)[at]
    x = raw.view(cache.dtype).double()
    return x if s[name + "_scale"] is None else x * s[name + "_scale"].double()[:, None]


def _attend64(s):
    q = s["q"].double()
    out = torch.zeros_like(q)
    H, G = s["case"]["Hkv"], s["case"]["Hq"] // s["case"]["Hkv"]
    tokens, ctx = _count(s).tolist(), s["ctx_len"].tolist()
    # contiguous() of a view makes a copy: do it once
    for name in ("k_cache", "v_cache"):
        s[name] = s[name].contiguous()
    for b in range(len(ctx)):
        slots = torch.arange(ctx[b] + tokens[b], device=q.device)
        k, v = (_slots64(s, n, b, slots).transpose(0, 1) for n in "kv")  # [H, S, D]
        rule = None if s["mask"] is None else s["mask"][b].tolist()
        for t in range(tokens[b]):
            seen = torch.ones_like(slots, dtype=torch.bool)
            for i in range(tokens[b]):
                seen[ctx[b] + i] = i <= t if rule is None else bool((rule[t] >> i) & 1)
            if not bool(seen.any()):
                continue
            z = torch.matmul(q[b, t].view(H, G, -1), k[:, seen].transpose(1, 2)) * s["scale"]  # [H, G, S]
            w = torch.exp(z - torch.logsumexp(z, -1, keepdim=True))
            out[b, t] = torch.matmul(w, v[:, seen]).view(H * G, -1)
    return out


def _append64(s):
    case, dev = s["case"], s["q"].device
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    r, page = case["rot"], case["page"]
    tokens, ctx = _count(s).tolist(), s["ctx_len"].tolist()
    for b in range(case["B"]):
        n = tokens[b]
        slots = ctx[b] + torch.arange(n, device=dev)
        at = slots if s["positions"] is None else s["positions"][b, :n].long()

        def turned(x):
            x = x[b, :n].double().clone()
            if r:
                angle = (s["cos"][at].double() + 1j * s["sin"][at].double())[:, None]
                first, second = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
                y = torch.complex(x[..., first], x[..., second]) * angle
                x[..., first], x[..., second] = y.real, y.imag
            return x

        out[b, :n] = turned(s["q"])
        for cache, x, scale in ((caches[0], turned(s["k"]), s["k_scale"]), (caches[1], s["v"][b, :n].double(), s["v_scale"])):
            if scale is not None:
                x = (x / scale.double()[:, None]).clamp(-F8_MAX, F8_MAX)
            cache[s["pages"][b].long()[slots // page], slots % page] = x
    return [out, *caches]


def _keep64(s):
    page, done = s["case"]["page"], []
    ctx, path, kept, pages = s["ctx_len"].tolist(), s["path"].tolist(), s["n_keep"].tolist(), s["pages"].tolist()
    for cache in (s["k_cache"].double(), s["v_cache"].double()):
        for b, n in enumerate(kept):
            for i in range(n):
                at, to = ctx[b] + path[b][i], ctx[b] + i
                if at != to:
                    cache[:, pages[b][to // page], to % page] = cache[:, pages[b][at // page], at % page]
        done.append(cache)
    return done


def _logits64(s):
    out = s["out"].double()
    V, dev = out.shape[-1], out.device
    tokens, held, prompt = _count(s).tolist(), s["history_len"].tolist(), s["prompt_len"].tolist()
    bit = torch.arange(V, device=dev)
    for b, n in enumerate(tokens):
        ids = s["history"][b].long()
        before = torch.bincount(ids[: prompt[b]], minlength=V) > 0
        count = torch.bincount(ids[prompt[b]: held[b]], minlength=V)
        for t in range(n):
            if t:
                count[s["draft"][b, t - 1].long()] += 1
            z = s["logits"][b, t].double()
            if s["repetition"] is not None:
                r, f, p = (s[k][b].double() for k in ("repetition", "frequency", "presence"))
                z = torch.where(before | (count > 0), torch.minimum(z * r, z / r) if r >= 1 else torch.maximum(z * r, z / r), z)
                z = z - f * count - p * (count > 0)
            if s["bias"] is not None:
                z[s["bias_ids"][b].long()] += s["bias"][b].double()
            if s["mask"] is not None:
                z[((s["mask"][b, t].long()[bit // 32] >> (bit % 32)) & 1) == 0] = -math.inf
            out[b, t] = z
    return out
