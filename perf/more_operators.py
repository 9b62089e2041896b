"""Operators of long contexts, at the sizes they are measured at: an 8-bit cache with a scale per page and head, and
eviction from a paged cache by accumulated attention weight.

A cache of E4M3 codes whose scales follow the data: ``kv_append`` sets a page's scale from what goes into it (and
rescales what is there where it grows), ``paged_attention`` reads it, ``kv_keep`` moves a verified branch within it.
``kv_weigh`` adds up what attention gives every entry, ``kv_select`` picks the entries that stay within a budget, and
``kv_move`` brings them together.  Weights and positions of the entries lie in pages, [num_pages, heads, page_size].

``run`` computes them in elementary torch operations, or, where ``own`` is true, through this package's calls.
"""
from __future__ import annotations

import math

import torch

own = False

F8 = torch.float8_e4m3fn
F8_MAX = 448.0
ROPE_BASE = 10000.0
LEAST, MOST = -24, 24  # a page's scale is a power of two in 2^LEAST .. 2^MOST


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # one stream decoding one token: all launch latency
        dict(name="attend one token", op="attend", B=1, T=1, Hq=8, Hkv=2, D=64, page=16, ctx_lo=515, ctx_hi=515,
             cache="pages", chains=0, ragged=False, layout="slot", lse=False),
        # a serving batch of 64 requests with 6 drafts each, whose entries are then weighed: the cache at memory speed
        dict(name="attend batch", op="attend", B=64, T=7, Hq=32, Hkv=8, D=128, page=32, ctx_lo=1000, ctx_hi=16000,
             cache="pages", chains=0, ragged=True, layout="head", lse=True),
        # the drafted tokens of a small batch
        dict(name="append drafts", op="append", B=8, T=6, Hq=32, Hkv=8, D=128, page=16, ctx_lo=0, ctx_hi=4001,
             cache="pages", chains=0, ragged=True, layout="slot", interleaved=False, rot=128),
        # a chunk of prompts
        dict(name="append prompts", op="append", B=4, T=2047, Hq=32, Hkv=8, D=128, page=32, ctx_lo=1, ctx_hi=130,
             cache="pages", chains=0, ragged=True, layout="head", interleaved=True, rot=64),
        # one layer of one small batch: a branch of two chains
        dict(name="keep one layer", op="keep", L=1, B=4, T=9, Hkv=8, D=128, page=16, ctx_lo=17, ctx_hi=300,
             cache="pages", chains=2, layout="slot"),
        # every layer of a serving batch at once
        dict(name="keep all layers", op="keep", L=32, B=64, T=17, Hkv=8, D=128, page=16, ctx_lo=30, ctx_hi=200,
             cache="pages", chains=4, layout="head"),
        # the drafts of a small batch over a bf16 cache, contexts from empty to a few thousand tokens
        dict(name="weigh drafts", op="weigh", B=8, T=6, Hq=32, Hkv=8, D=128, page=16, ctx_lo=0, ctx_hi=4001,
             cache="bf16", chains=0, ragged=True, layout="slot"),
        # a serving batch over the 8-bit cache: the keys are read at memory speed
        dict(name="weigh batch", op="weigh", B=64, T=7, Hq=32, Hkv=8, D=128, page=32, ctx_lo=1000, ctx_hi=16000,
             cache="pages", chains=0, ragged=True, layout="head"),
        # a small batch a few tokens over its budget, some requests still under it
        dict(name="select a few", op="select", L=1, B=8, Hkv=8, page=16, ctx_lo=700, ctx_hi=1030, budget=1024, first=4,
             recent=256),
        # four layers of long contexts cut to a quarter
        dict(name="select long", op="select", L=4, B=16, Hkv=8, page=64, ctx_lo=30000, ctx_hi=65003, budget=16384, first=4,
             recent=4096),
        # a small batch a few tokens over its budget, 8-bit
        dict(name="move a few", op="move", L=1, B=8, Hkv=8, D=128, page=16, ctx_lo=700, ctx_hi=1030, budget=1024,
             cache="pages", layout="slot"),
        # long contexts cut to half in an 8-bit cache
        dict(name="move half", op="move", L=1, B=32, Hkv=8, D=128, page=32, ctx_lo=8000, ctx_hi=16000, budget=6000,
             cache="pages", layout="head"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "append", "keep", "weigh", "weigh", "select", "move"))
    c = dict(op=op, Hkv=rng.choice((1, 2, 4, 5, 8)), page=rng.choice((8, 16, 32, 64, 128, 256)))
    if op == "select":
        L, B = _log_int(rng, 1, 8), _log_int(rng, 1, 64)
        hi = _log_int(rng, 2, max(2, min(131072, int(2.4e7 / (L * B * c["Hkv"])))))
        return dict(c, L=L, B=B, ctx_lo=rng.randint(0, hi), ctx_hi=hi, budget=rng.randint(1, hi), first=rng.choice((0, 1, 4)),
                    recent=rng.choice((0, 1, 32, hi // 8)))
    c.update(D=rng.choice((64, 128)), cache="pages", layout=rng.choice(("slot", "head")))
    slot_bytes = c["Hkv"] * c["D"] * 2
    if op == "move":
        c["cache"] = rng.choice(("pages", "pages", "bf16", "e4m3"))
        L, B = _log_int(rng, 1, 4), _log_int(rng, 1, 64)
        hi = _log_int(rng, 2, max(2, min(65536, int(2.5e8 / (L * B * slot_bytes)))))
        return dict(c, L=L, B=B, ctx_lo=rng.randint(0, hi), ctx_hi=hi, budget=rng.randint(1, hi))
    group = rng.choice((1, 2, 3, 4, 7, 8, 16))
    chains = 0
    T = rng.choice((1, 1, 2, 3, 4, 5, 6, 7, 8, 9, 13, 17))
    if op == "keep" or rng.random() < 0.25:
        chains = rng.randint(2, 4)
        T = 1 + chains * rng.randint(1, 12)
    if op == "keep":
        L = _log_int(rng, 1, 40)
        B = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, max(1, min(2000, int(3e8 / (L * B * slot_bytes)))))
        return dict(c, L=L, B=B, T=T, chains=chains, ctx_lo=rng.randint(0, hi), ctx_hi=hi)
    if op == "append":
        if not chains and rng.random() < 0.4:
            T = _log_int(rng, 17, 4000)
        B = _log_int(rng, 1, max(1, min(256, int(1.4e8 / (T * (group + 2) * c["Hkv"] * c["D"] * 4)))))
        hi = _log_int(rng, 1, max(1, min(4000, int(2.5e8 / (B * slot_bytes)))))
        return dict(c, B=B, T=T, Hq=group * c["Hkv"], chains=chains, ctx_lo=rng.randint(0, hi), ctx_hi=hi,
                    ragged=rng.random() < 0.5, interleaved=rng.random() < 0.5, rot=rng.choice((0, 32, 64, c["D"])))
    if op == "weigh":
        c["cache"] = rng.choice(("pages", "pages", "bf16", "e4m3"))
    most = min(5e8 / slot_bytes, 2e10 / (4 * T * group * c["Hkv"] * c["D"]))  # cache slots of all requests together
    hi = _log_int(rng, 1, max(1, min(131072, int(most))))
    B = _log_int(rng, 1, max(1, min(256, int(most / hi))))
    c = dict(c, B=B, T=T, Hq=group * c["Hkv"], chains=chains, ctx_lo=rng.randint(0, hi), ctx_hi=hi, ragged=rng.random() < 0.5)
    return dict(c, lse=rng.random() < 0.5) if op == "attend" else c


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
    """A pool of pages [layers, pages, page, heads, D] as views of the asked memory order, with its scales.  A page's
    codes fill its range as kv_append leaves them: a standard deviation of 100, pages a factor of 2 or 4 apart."""
    dev, H, D, ps = "cuda", case["Hkv"], case["D"], case["page"]
    shape = (layers, num_pages, H, ps, D) if case["layout"] == "head" else (layers, num_pages, ps, H, D)
    pool, scales = [], []
    for _ in range(2):
        x = torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(0.0, 100.0 if case["cache"] == "pages" else 1.0, generator=g)
        if case["cache"] != "bf16":
            x = x.clamp_(-F8_MAX, F8_MAX).to(F8)
        pool.append(x.transpose(2, 3) if case["layout"] == "head" else x)
        if case["cache"] == "pages":
            scales.append(torch.exp2(torch.randint(-8, -5, (layers, num_pages, H), generator=g, device=dev).float()))
        else:
            scales.append(torch.rand(H, generator=g, device=dev) * 0.5 + 0.5 if case["cache"] == "e4m3" else None)
    return pool + scales


def _record(layers, num_pages, case, g):
    """Accumulated weights with a long tail, [layers, pages, heads, page]."""
    u = torch.rand((layers, num_pages, case["Hkv"], case["page"]), generator=g, device="cuda")
    return torch.exp(3.0 * u * u) * (u * 0.01 + 1e-4)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    B, op, page, H = case["B"], case["op"], case["page"], case["Hkv"]
    T = case.get("T", 0)
    i32 = dict(dtype=torch.int32, device=dev)
    order = torch.randperm(B, generator=g, device=dev)
    s = dict(case=case)
    s["t_per_row"] = torch.tensor(_tokens(case), **i32)[order] if case.get("ragged") else None
    maxp = -(-(case["ctx_hi"] + T) // page)
    num_pages = B * maxp + 3
    s["pages"] = torch.randperm(num_pages, generator=g, device=dev)[: B * maxp].to(torch.int32).view(B, maxp)
    s["ctx_len"] = torch.tensor(_spread(case["ctx_lo"], case["ctx_hi"], B), **i32)[B - 1 - order]
    layers = case.get("L", 1)
    if op in ("select", "move"):
        s["weight"] = _record(layers, num_pages, case, g)
        s["position"] = torch.empty((layers, num_pages, H, page), **i32)
        # entries of earlier evictions lie in no order, and a request has seen more tokens than it holds
        s["seen"] = s["ctx_len"] + s["ctx_len"] // 3 + 5
        u = torch.rand((layers, B, H, maxp * page), generator=g, device=dev)
        u = torch.where(torch.arange(maxp * page, device=dev) < s["ctx_len"][:, None, None], u, 2.0)
        place = (u.argsort(-1).argsort(-1) * 4 // 3).to(torch.int32)
        s["position"].copy_(torch.randint(0, 1 << 20, s["position"].shape, generator=g, device=dev))
        s["position"][:, s["pages"].long()] = place.view(layers, B, H, maxp, page).transpose(2, 3)
        s["budget"] = torch.full((B,), case["budget"], **i32)
        n = max(1, maxp * page // 2)
        s["source"], s["target"] = (torch.full((layers, B, H, n), -1, **i32) for _ in range(2))
        s["moves"], s["new_len"] = torch.zeros((layers, B, H), **i32), torch.zeros(B, **i32)
        if op == "select":
            return s
        # what a selection that goes by the weights alone gives
        s["source"], s["target"], s["moves"], s["new_len"] = _chosen(s, 0, 0)
    k, v, ks, vs = _cache(case, layers, num_pages, g)
    if op in ("keep", "move"):
        s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = k, v, ks, vs
        if op == "move":
            return s
        K = (T - 1) // case["chains"]
        chain = torch.randint(0, case["chains"], (B, 1), generator=g, device=dev)
        s["path"] = torch.cat([torch.zeros_like(chain), 1 + chain * K + torch.arange(K, device=dev)], 1).to(torch.int32)
        s["n_keep"] = torch.tensor(_spread(1, K + 1, B), **i32)[order]  # the root and the accepted drafts
        return s
    s["k_cache"], s["v_cache"] = k[0], v[0]
    s["k_scale"], s["v_scale"] = (ks[0], vs[0]) if case["cache"] == "pages" else (ks, vs)
    D, Hq = case["D"], case["Hq"]
    normal = lambda h, sd: torch.empty((B, T, h, D), dtype=torch.bfloat16, device=dev).normal_(0.0, sd, generator=g)  # noqa: E731
    s["positions"] = s["mask"] = None
    if case["chains"]:
        depth, bits = _tree(T, case["chains"])
        s["mask"] = torch.tensor(bits, dtype=torch.int64, device=dev).expand(B, T).contiguous()
        s["positions"] = s["ctx_len"][:, None] + torch.tensor(depth, **i32)
    if op in ("attend", "weigh"):
        s["q"] = normal(Hq, 1.5)
        s["scale"] = 1.0 / math.sqrt(D)
        s["lse"] = torch.full((B, T, Hq), -math.inf, device=dev)
        if op == "weigh":
            del s["v_cache"], s["v_scale"]
            s["lse"] = _sums(s)
            s["weight"] = _record(1, num_pages, case, g)[0]
            s["position"] = torch.zeros((num_pages, H, page), **i32)
        return s
    # one projection's output holds the heads of q, k and v side by side
    qkv = normal(Hq + 2 * H, 1.5)
    s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq: Hq + H], qkv[:, :, Hq + H:]
    s["cos"] = s["sin"] = None
    if case["rot"]:
        n = case["ctx_hi"] + T
        freq = ROPE_BASE ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
        angle = torch.arange(n, device=dev, dtype=torch.float64)[:, None] * freq
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    s["out"] = torch.zeros((B, T, Hq, D), dtype=torch.bfloat16, device=dev)
    return s


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        import speculative_decoding_rejection_verify_gb300 as sv
        if op == "attend":
            out = sv.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["ctx_len"], s["t_per_row"],
                                     mask=s["mask"], scale=s["scale"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                     lse=s["lse"] if s["case"]["lse"] else None)
            return [out, s["lse"]] if s["case"]["lse"] else out
        if op == "append":
            q = sv.kv_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["pages"], s["ctx_len"], s["cos"],
                             s["sin"], s["t_per_row"], positions=s["positions"], interleaved=s["case"]["interleaved"],
                             k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"])
            return [q, s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]
        if op == "keep":
            sv.kv_keep(s["k_cache"], s["v_cache"], s["pages"], s["ctx_len"], s["path"], s["n_keep"],
                       k_scale=s["k_scale"], v_scale=s["v_scale"])
            return [s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]
        if op == "weigh":
            sv.kv_weigh(s["q"], s["k_cache"], s["pages"], s["ctx_len"], s["lse"], s["weight"], s["position"],
                        t_per_row=s["t_per_row"], mask=s["mask"], positions=s["positions"], scale=s["scale"],
                        k_scale=s["k_scale"])
            return [s["weight"], s["position"]]
        if op == "select":
            return list(sv.kv_select(s["weight"], s["position"], s["pages"], s["ctx_len"], s["budget"], seen=s["seen"],
                                     first=s["case"]["first"], recent=s["case"]["recent"],
                                     out=(s["source"], s["target"], s["moves"], s["new_len"])))
        paged = s["case"]["cache"] == "pages"
        sv.kv_move(s["k_cache"], s["v_cache"], s["pages"], s["new_len"], s["source"], s["target"], s["moves"],
                   k_scale=s["k_scale"] if paged else None, v_scale=s["v_scale"] if paged else None, weight=s["weight"],
                   position=s["position"])
        return _moved(s)
    return {"attend": _attend, "append": _append, "keep": _keep, "weigh": _weigh, "select": _select, "move": _move}[op](s)


def _moved(s):
    scales = [s["k_scale"], s["v_scale"]] if s["case"]["cache"] == "pages" else []
    return [s["k_cache"], s["v_cache"], *scales, s["weight"], s["position"]]


def _count(s):
    """[B] valid new tokens."""
    t = s["t_per_row"]
    return t if t is not None else torch.full((s["case"]["B"],), s["case"]["T"], dtype=torch.int32, device="cuda")


def _gather(s, name):
    """The cache of every request side by side, [B, slots, heads, D] in 32 bits."""
    cache, scale, pages = s[name + "_cache"], s[name + "_scale"], s["pages"].long()
    if cache.dtype != F8:
        return cache[pages].flatten(1, 2).float()
    x = cache.view(torch.uint8)[pages].view(F8).float()  # [B, pages, page, heads, D]
    x = x * (scale[pages][:, :, None, :, None] if s["case"]["cache"] == "pages" else scale[:, None])
    return x.flatten(1, 2)


def _sees(s, S):
    """[B, T, S]: which slots each new token attends to."""
    tb, ctx, t = _count(s), s["ctx_len"], torch.arange(s["case"]["T"], device="cuda")
    new = torch.arange(S, device="cuda") - ctx[:, None]  # which new token a slot holds, negative in the context
    if s["mask"] is None:
        sees = new[:, None] <= t[:, None]
    else:
        sees = (new[:, None] < 0) | ((s["mask"][:, :, None] >> new[:, None].clamp(0, 63)) & 1).bool()
    return sees & (new < tb[:, None])[:, None] & (t < tb[:, None])[:, :, None]


def _scores(s, k):
    """[B, heads, group, T, S], -inf where a row does not attend."""
    q, S = s["q"], k.shape[1]
    B, T, Hq, D = q.shape
    H = k.shape[2]
    rows = q.float().view(B, T, H, Hq // H, D).permute(0, 2, 3, 1, 4).reshape(B, H, -1, D)
    z = torch.matmul(rows, k.permute(0, 2, 3, 1)).view(B, H, Hq // H, T, S) * s["scale"]
    return z.masked_fill(~_sees(s, S)[:, None, None], -math.inf)


def _attend(s):
    q, tb, ctx = s["q"], _count(s), s["ctx_len"]
    B, T, Hq, D = q.shape
    k, v = _gather(s, "k"), _gather(s, "v")
    S, H = k.shape[1:3]
    held = torch.arange(S, device=q.device) < (ctx + tb)[:, None]
    v = torch.where(held[:, :, None, None], v, 0.0)
    z = _scores(s, k)
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - torch.where(m == -math.inf, 0.0, m))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e.view(B, H, -1, S), v.permute(0, 2, 1, 3)).view(B, H, Hq // H, T, D)
    o = torch.where(total > 0, o / total, 0.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(q.dtype)
    if not s["case"]["lse"]:
        return o
    s["lse"].copy_((m + torch.log(total))[..., 0].permute(0, 3, 1, 2).reshape(B, T, Hq))
    return [o, s["lse"]]


def _weigh(s):
    """Weights and positions of the slots that hold tokens."""
    k = _gather(s, "k")
    B, S, H, D = k.shape
    T, G = s["case"]["T"], s["case"]["Hq"] // H
    lse = s["lse"].view(B, T, H, G).permute(0, 2, 3, 1)[..., None]
    w = torch.exp(_scores(s, k) - torch.where(lse == -math.inf, math.inf, lse)).sum((2, 3))  # [B, heads, S]
    slot, page = torch.arange(S, device=k.device), s["case"]["page"]
    ctx, held = s["ctx_len"], slot < (s["ctx_len"] + _count(s))[:, None]
    b, at = held.nonzero(as_tuple=True)
    where, fresh = (s["pages"].long()[b, at // page], slice(None), at % page), at >= ctx[b]
    s["weight"][where] = torch.where(fresh[:, None], 0.0, s["weight"][where]) + w[b, :, at]
    b, at = b[fresh], at[fresh]
    new = at - ctx[b]
    value = at if s["positions"] is None else s["positions"][b, new]
    s["position"][s["pages"].long()[b, at // page], :, at % page] = value.to(torch.int32)[:, None]
    return [s["weight"], s["position"]]


def _rotate(x, cos, sin, interleaved):
    r = 2 * cos.shape[-1]
    cos, sin = cos[:, :, None], sin[:, :, None]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., : r // 2], x[..., r // 2: r])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _need(most):
    """The smallest power of two s in its range with most <= 448 s."""
    m, e = torch.frexp(most)  # most = m 2^e, m in [0.5, 1), and 448 = 0.875 * 2^9
    e = torch.where(most > 0, e - 9 + (m > 0.875), LEAST).clamp(LEAST, MOST)
    return torch.ldexp(torch.ones_like(most), e)


def _most(x):
    """The largest finite |x| of every head vector."""
    x = x.abs()
    return torch.where(torch.isfinite(x), x, 0.0).amax(-1)


def _codes(x):
    return x.clamp(-F8_MAX, F8_MAX).to(F8).view(torch.uint8)


def _append(s):
    B, T, page = s["case"]["B"], s["case"]["T"], s["case"]["page"]
    ctx, dev = s["ctx_len"].long(), s["q"].device
    t = torch.arange(T, device=dev)
    slot = ctx[:, None] + t
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if s["cos"] is not None:
        at = slot if s["positions"] is None else s["positions"].long()
        cos, sin = s["cos"][at], s["sin"][at]
        q, k = (_rotate(x, cos, sin, s["case"]["interleaved"]) for x in (q, k))
    valid = t < _count(s)[:, None]
    s["out"].copy_(torch.where(valid[:, :, None, None], q, 0.0))
    place = torch.gather(s["pages"].long(), 1, slot // page)
    where = place[valid], (slot % page)[valid]
    # the page that the context ends in keeps what it holds
    inner = ctx % page
    ends = torch.gather(s["pages"].long(), 1, (ctx // page)[:, None].clamp(max=s["pages"].shape[1] - 1))[:, 0]
    holds = (inner > 0) & (_count(s) > 0)
    row = torch.arange(page, device=dev)
    for name, x in (("k", k), ("v", v)):
        codes, scale = s[name + "_cache"].view(torch.uint8), s[name + "_scale"]
        most = torch.full_like(scale, -1.0)
        most.index_reduce_(0, where[0], _most(x[valid]), "amax")
        old, fresh = scale[ends[holds]], _need(most.clamp(min=0.0))
        new = torch.where(most >= 0, fresh, scale)
        new[ends[holds]] = torch.maximum(old, fresh[ends[holds]])
        grown = new[ends[holds]] > old
        pages = codes[ends[holds]]  # [requests, page, heads, D]
        again = _codes(pages.view(F8).float() * (old / new[ends[holds]])[:, None, :, None])
        change = grown[:, None, :, None] & (row < inner[holds][:, None])[:, :, None, None]
        codes[ends[holds]] = torch.where(change, again, pages)
        codes[where] = _codes(x[valid] / new[where[0]][:, :, None])
        scale.copy_(new)
    return [s["out"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]


def _shift(s, layer, request, head, source, target, stays):
    """Entries move from source to target slots (one per element of the index lists) in an 8-bit cache with page scales;
    stays [pages, page] or [layers, pages, page, heads]: what its page's new scale has to hold as well."""
    pages, page = s["pages"].long(), s["case"]["page"]
    at = (layer, pages[request, source // page], source % page, head)
    to = (layer, pages[request, target // page], target % page, head)
    for name in "kv":
        codes, scale = s[name + "_cache"].view(torch.uint8), s[name + "_scale"]
        x = codes[at].view(F8).float() * scale[layer, at[1], head][:, None]
        most = torch.full_like(scale, -1.0).view(-1)
        flat = (layer * scale.shape[1] + to[1]) * scale.shape[2] + head
        most = most.index_reduce_(0, flat, _most(x), "amax").view_as(scale)
        new = torch.where(most >= 0, torch.maximum(scale, _need(most.clamp(min=0.0))), scale)
        change = (new > scale)[:, :, None, :, None] & stays[..., None]
        ratio = (scale / new)[:, :, None, :, None]
        codes.copy_(torch.where(change, _codes(codes.view(F8).float() * ratio), codes))
        codes[to] = _codes(x / new[layer, to[1], head][:, None])
        scale.copy_(new)


def _held(s, end):
    """[num_pages, page]: whether a row holds one of the slots < end[b] of a request."""
    page, (B, n) = s["case"]["page"], s["pages"].shape
    held = torch.zeros((s["k_cache"].shape[1], page), dtype=torch.bool, device=end.device)
    slot = torch.arange(n * page, device=end.device).view(n, page)
    held[s["pages"].long()] = slot < end[:, None, None]
    return held


def _keep(s):
    path, ctx = s["path"].long(), s["ctx_len"].long()
    L, H, dev, page = s["case"]["L"], s["case"]["Hkv"], path.device, s["case"]["page"]
    i = torch.arange(path.shape[1], device=dev)
    b, j = ((i < s["n_keep"][:, None]) & (path != i)).nonzero(as_tuple=True)
    source, target = ctx[b] + path[b, j], ctx[b] + j
    stays = _held(s, s["ctx_len"] + s["n_keep"])
    stays[s["pages"].long()[b, target // page], target % page] = False
    n = b.numel()
    every = lambda x: x.repeat(L * H)  # noqa: E731
    layer = torch.arange(L, device=dev).repeat_interleave(n * H)
    head = torch.arange(H, device=dev).repeat_interleave(n).repeat(L)
    _shift(s, layer, every(b), head, every(source), every(target), stays[None, :, :, None])
    return [s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]


def _chosen(s, first, recent):
    """(source, target, moves, new_len) of a selection."""
    pages, ctx = s["pages"].long(), s["ctx_len"]
    side = lambda x: x[:, pages].transpose(2, 3).flatten(3)  # noqa: E731  [layers, B, heads, slots]
    w, p = side(s["weight"]), side(s["position"])
    slot = torch.arange(w.shape[-1], device=w.device)
    w = torch.where((p < first) | (p >= (s["seen"] - recent)[:, None, None]), math.inf, torch.nan_to_num(w, nan=-math.inf, posinf=math.inf, neginf=-math.inf))
    here = (slot < ctx[:, None])[:, None]
    # slots behind the context come last: a sort by weight, ties by slot, then by whether there is an entry
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices
    absent = ~torch.gather(here.expand(w.shape), -1, order)
    order = torch.gather(order, -1, torch.sort(absent.to(torch.uint8), dim=-1, stable=True).indices)
    m = torch.minimum(ctx, s["budget"].clamp(min=0))
    rank = torch.empty_like(order).scatter_(-1, order, slot.expand(order.shape).contiguous())
    kept = here & (rank < m[:, None, None])
    below = slot < m[:, None, None]
    out = []
    for chosen, before in ((kept & ~below, s["source"]), (~kept & below, s["target"])):
        index = chosen.nonzero(as_tuple=True)
        place = (chosen.cumsum(-1) - 1)[index]
        x = before.clone()
        x[index[0], index[1], index[2], place] = index[3].to(torch.int32)
        out.append(x)
    return [*out, (kept & ~below).sum(-1).to(torch.int32), m.to(torch.int32)]


def _select(s):
    got = _chosen(s, s["case"]["first"], s["case"]["recent"])
    for name, x in zip(("source", "target", "moves", "new_len"), got):
        s[name].copy_(x)
    return [s["source"], s["target"], s["moves"], s["new_len"]]


def _move(s):
    n = torch.arange(s["source"].shape[-1], device="cuda") < s["moves"][..., None]
    layer, request, head, _ = n.nonzero(as_tuple=True)
    source, target = s["source"][n].long(), s["target"][n].long()
    pages, page = s["pages"].long(), s["case"]["page"]
    at = (layer, pages[request, source // page], source % page, head)
    to = (layer, pages[request, target // page], target % page, head)
    if s["case"]["cache"] == "pages":
        stays = _held(s, s["new_len"])[None, :, :, None].expand(s["k_cache"].shape[:4]).clone()
        stays[to] = False
        _shift(s, layer, request, head, source, target, stays)
    else:
        for name in ("k_cache", "v_cache"):
            cache = s[name].view(torch.uint8) if s[name].dtype == F8 else s[name]
            cache[to] = cache[at]
    for x in (s["weight"], s["position"]):
        x = x.transpose(2, 3)
        x[to] = x[at]
    return _moved(s)


# ------------------------------------------------------------------------------------------------
# what a pass cannot do without, and the definition in 64 bits
# ------------------------------------------------------------------------------------------------
def _evicted(case):
    """Entries that move, of one head of one layer: what an even spread of the kept ones leaves behind the budget."""
    m = [min(n, case["budget"]) for n in _spread(case["ctx_lo"], case["ctx_hi"], case["B"])]
    return sum(k * (n - k) / n for k, n in zip(m, _spread(case["ctx_lo"], case["ctx_hi"], case["B"])) if n)


def work(case):
    B, op, H, page = case["B"], case["op"], case["Hkv"], case["page"]
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], B)
    if op == "select":
        lists = case["L"] * H
        return {"bytes": lists * (8 * sum(ctx) + 8 * _evicted(case) + 4 * B) + 4 * sum(-(-n // page) for n in ctx) + 12 * B,
                "flops": lists * sum(ctx)}
    es = 2 if case["cache"] == "bf16" else 1
    scaled = case["cache"] == "pages"
    D = case["D"]
    if op == "move":
        moved = case["L"] * H * _evicted(case)
        return {"bytes": moved * (2 * 2 * D * es + 2 * 8 + 8), "flops": 2 * moved * D if scaled else 0}
    slot = H * D
    if op == "keep":
        K = (case["T"] - 1) // case["chains"]
        moved = sum(n - 1 for n in _spread(1, K + 1, B)) * (case["chains"] - 1) / case["chains"]  # the first chain stays
        return {"bytes": case["L"] * moved * slot * 2 * 2 + case["L"] * B * H * 16 + B * (K + 3) * 4, "flops": case["L"] * moved * slot * 2}
    tokens = sum(_tokens(case))
    q = tokens * case["Hq"] * D * 2
    if op == "append":
        table = tokens * case["rot"] * 4
        pages = sum(-(-n // page) for n in _tokens(case))
        return {"bytes": 2 * q + tokens * slot * 2 * (2 + es) + table + pages * H * 8 + 8 * B,
                "flops": 3 * tokens * (case["Hq"] + H) * case["rot"] + 2 * tokens * slot * 2}
    pairs = [(c + t) for c, t in zip(ctx, _tokens(case)[::-1])]
    rows = sum(n * t for n, t in zip(pairs, _tokens(case)[::-1])) * case["Hq"]
    pages = sum(-(-n // page) for n in pairs)
    if op == "weigh":
        record = sum(8 * c + 8 * t for c, t in zip(ctx, _tokens(case)[::-1])) * H
        return {"bytes": q + tokens * case["Hq"] * 4 + sum(pairs) * slot * es + record + pages * (4 + (4 * H if scaled else 0)),
                "flops": 2 * rows * D + 3 * rows}
    return {"bytes": 2 * q + sum(pairs) * slot * 2 * es + pages * (4 + 8 * H) + (tokens * case["Hq"] * 4 if case["lse"] else 0),
            "flops": 4 * rows * D}


def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _attend64, "append": _append64, "keep": _keep64, "weigh": _weigh64, "select": _select64,
            "move": _move64}[case["op"]](s)


def _entries64(s, name, b, slots):
    """Cache entries of request b in 64 bits, [heads, slots, D]."""
    page = s["case"]["page"]
    p, r = s["pages"][b].long()[slots // page], slots % page
    cache, scale = s[name + "_cache"], s[name + "_scale"]
    x = cache[p, r].double() if cache.dtype != F8 else cache.view(torch.uint8)[p, r].view(F8).double()
    if scale is not None:
        x = x * (scale[p] if s["case"]["cache"] == "pages" else scale).double()[..., None]
    return x.transpose(0, 1)


def _rows64(s, names):
    """For every row that attends to something: (request, token, slots, scores [heads, group, slots], the named entries)."""
    q, H = s["q"].double(), s["case"]["Hkv"]
    tokens, ctx = _count(s).tolist(), s["ctx_len"].tolist()
    for b in range(len(ctx)):
        slots = torch.arange(ctx[b] + tokens[b], device=q.device)
        held = [_entries64(s, n, b, slots) for n in names]
        rule = None if s["mask"] is None else s["mask"][b].tolist()
        for t in range(tokens[b]):
            seen = list(range(ctx[b])) + [ctx[b] + i for i in range(tokens[b]) if (i <= t if rule is None else (rule[t] >> i) & 1)]
            if not seen:
                continue
            few = [i for i in range(tokens[b]) if ctx[b] + i not in seen[ctx[b]:]]
            at = slots if not few else slots[~torch.isin(slots, torch.tensor([ctx[b] + i for i in few], device=q.device))]
            z = torch.matmul(q[b, t].view(H, -1, q.shape[-1]), held[0][:, at].transpose(1, 2)) * s["scale"]
            yield b, t, at, z, held


def _sums(s):
    """log of the sum of exponentials of every row's scores, as the attention gives it."""
    B, T, Hq, _ = s["q"].shape
    H, page = s["case"]["Hkv"], s["case"]["page"]
    lse = torch.full((B, T, H, Hq // H), -math.inf, device=s["q"].device)
    whole = s
    for b in range(B):  # a request at a time: less memory, and only the slots that it has
        n = -(-(int(whole["ctx_len"][b]) + T) // page)
        s = {**whole, "case": {**whole["case"], "B": 1}, "q": whole["q"][b:b + 1], "pages": whole["pages"][b:b + 1, :n],
             "ctx_len": whole["ctx_len"][b:b + 1], "t_per_row": None if whole["t_per_row"] is None else whole["t_per_row"][b:b + 1],
             "mask": None if whole["mask"] is None else whole["mask"][b:b + 1]}
        lse[b] = torch.logsumexp(_scores(s, _gather(s, "k")), -1)[0].permute(2, 0, 1)
    return lse.view(B, T, Hq)


def _attend64(s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = s["lse"].double()
    for b, t, at, z, held in _rows64(s, "kv"):
        total = torch.logsumexp(z, -1)
        out[b, t] = torch.matmul(torch.exp(z - total[..., None]), held[1][:, at]).view(out.shape[2:])
        lse[b, t] = total.view(-1)
    return [out, lse] if s["case"]["lse"] else out


def _weigh64(s):
    weight, position, page = s["weight"].double(), s["position"], s["case"]["page"]
    tokens, ctx = _count(s).tolist(), s["ctx_len"].tolist()
    for b, c in enumerate(ctx):
        for t in range(tokens[b]):
            p, r = s["pages"][b, (c + t) // page].long(), (c + t) % page
            weight[p, :, r] = 0.0
            position[p, :, r] = c + t if s["positions"] is None else s["positions"][b, t]
    for b, t, at, z, _ in _rows64(s, "k"):
        lse = s["lse"][b, t].double().view(z.shape[0], -1, 1)
        weight[s["pages"][b].long()[at // page], :, at % page] += torch.exp(z - lse).sum(1).T
    return [weight, position]


def _need64(most):
    return 0.0 if most is None else 2.0 ** max(LEAST, min(MOST, math.ceil(math.log2(most / F8_MAX)))) if most > 0 else 2.0 ** LEAST


def _put64(values, scale, page, head, rows, x, stays):
    """Entries x [rows, D] go into one page of `values` (the codes' values, [pages, page, heads, D]) in 64 bits."""
    fine = x[torch.isfinite(x)].abs()
    need = _need64(float(fine.max()) if fine.numel() else 0.0)
    old = float(scale[page, head])
    new = need if stays is None else max(old, need)
    if stays is not None and new > old:
        values[page, stays, head] *= old / new
    values[page, rows, head] = (x / new).clamp(-F8_MAX, F8_MAX)
    scale[page, head] = new


def _append64(s):
    case, dev = s["case"], s["q"].device
    tokens, ctx, r, page = _count(s).tolist(), s["ctx_len"].tolist(), case["rot"], case["page"]
    if sum(tokens) * case["Hkv"] > 20000 * page:
        return None  # too many pages to go through one by one
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    caches, scales = [s[n].double() for n in ("k_cache", "v_cache")], [s[n].double() for n in ("k_scale", "v_scale")]
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
        for cache, scale, x in zip(caches, scales, (turned(s["k"]), s["v"][b, :n].double())):
            for p in range(ctx[b] // page, (ctx[b] + n - 1) // page + 1 if n else 0):
                here = (slots // page) == p
                stays = torch.arange(ctx[b] % page, device=dev) if p * page < ctx[b] else None
                for h in range(case["Hkv"]):
                    _put64(cache, scale, int(s["pages"][b, p]), h, slots[here] % page, x[here, h], stays)
    return [out, *caches, *scales]


def _shift64(s, moves, stays):
    """moves: of every (layer, request, head) its (sources, targets); stays(b): the slots whose entries keep their place."""
    page, out = s["case"]["page"], []
    if sum(len(x) for x in moves.values()) > 4000:
        return None
    for name in "kv":
        values, scale = s[name + "_cache"].double(), s[name + "_scale"].double()
        codes, before = values.clone(), scale.clone()
        for (layer, b, h), pairs in moves.items():
            place = lambda n: (int(s["pages"][b, n // page]), n % page)  # noqa: E731
            for p in sorted({t // page for _, t in pairs}):
                mine = [(a, t) for a, t in pairs if t // page == p]
                x = torch.stack([codes[layer, place(a)[0], place(a)[1], h] * before[layer, place(a)[0], h] for a, _ in mine])
                taken = {t for _, t in mine}
                rest = torch.tensor([n % page for n in range(p * page, p * page + page) if n in stays(b) and n not in taken], dtype=torch.long, device="cuda")
                _put64(values[layer], scale[layer], place(mine[0][1])[0], h, torch.tensor([t % page for t in sorted(taken)], device="cuda"), x, rest)
        out.append((values, scale))
    return [out[0][0], out[1][0], out[0][1], out[1][1]]


def _keep64(s):
    ctx, path, kept = s["ctx_len"].tolist(), s["path"].tolist(), s["n_keep"].tolist()
    moves = {(layer, b, h): [(ctx[b] + p, ctx[b] + i) for i, p in enumerate(path[b][:n]) if p != i]
             for layer in range(s["case"]["L"]) for b, n in enumerate(kept) for h in range(s["case"]["Hkv"])}
    return _shift64(s, {k: v for k, v in moves.items() if v}, lambda b: range(ctx[b] + kept[b]))


def _select64(s):
    if s["weight"].numel() > 3e6:
        return None
    page, (L, B, H, _) = s["case"]["page"], s["source"].shape
    weight, position = s["weight"].double().cpu(), s["position"].cpu()
    ctx, seen, budget, pages = (s[n].tolist() for n in ("ctx_len", "seen", "budget", "pages"))
    for layer in range(L):
        for b in range(B):
            m = min(ctx[b], max(budget[b], 0))
            s["new_len"][b] = m
            for h in range(H):
                w, p = (x[layer][pages[b], h].flatten().tolist() for x in (weight, position))
                far = [math.inf if p[n] < s["case"]["first"] or p[n] >= seen[b] - s["case"]["recent"] else w[n] for n in range(ctx[b])]
                kept = set(sorted(range(ctx[b]), key=lambda n: (-far[n], n))[:m])
                source, target = sorted(n for n in kept if n >= m), [n for n in range(m) if n not in kept]
                s["moves"][layer, b, h] = len(source)
                s["source"][layer, b, h, : len(source)] = torch.tensor(source, dtype=torch.int32)
                s["target"][layer, b, h, : len(target)] = torch.tensor(target, dtype=torch.int32)
    return [s["source"], s["target"], s["moves"], s["new_len"]]


def _move64(s):
    page, count = s["case"]["page"], s["moves"].tolist()
    moves, end = {}, s["new_len"].tolist()
    if s["moves"].sum() > 4000:
        return None
    for layer, rows in enumerate(count):
        for b, row in enumerate(rows):
            for h, n in enumerate(row):
                if n:
                    moves[layer, b, h] = list(zip(s["source"][layer, b, h, :n].tolist(), s["target"][layer, b, h, :n].tolist()))
    if s["case"]["cache"] == "pages":
        done = _shift64(s, moves, lambda b: range(end[b]))
    else:
        done = [s["k_cache"].double(), s["v_cache"].double()]
        for (layer, b, h), pairs in moves.items():
            for a, t in pairs:
                for x in done:
                    x[layer, s["pages"][b, t // page].long(), t % page, h] = x[layer, s["pages"][b, a // page].long(), a % page, h]
    weight, position = s["weight"].double(), s["position"].clone()
    for (layer, b, h), pairs in moves.items():
        for a, t in pairs:
            for x in (weight, position):
                x[layer, s["pages"][b, t // page].long(), h, t % page] = x[layer, s["pages"][b, a // page].long(), h, a % page]
    return [*done, weight, position]
