"""Inputs and 64-bit references of the decode-step operators' tests.

The references follow the formulas one token, head and slot at a time, in float64 on the CPU, and
return beside each result what its error bound is made of.
"""
from __future__ import annotations

import math

import numpy as np
import torch

U_BF16 = 2.0 ** -8     # unit roundoff of bfloat16 (8 significant bits)
U_F32 = 2.0 ** -24
U_E4M3 = 2.0 ** -4     # 4 significant bits
F8 = torch.float8_e4m3fn


def pool(num_pages, page, heads, D, dtype, layout, g, layers=None, fill=None):
    """Two cache tensors [num_pages, page, heads, D] (with layers in front if asked) on the CPU."""
    lead = () if layers is None else (layers,)
    shape = lead + ((num_pages, heads, page, D) if layout == "head" else (num_pages, page, heads, D))
    out = []
    for _ in range(2):
        x = torch.randn(shape, generator=g) if fill is None else torch.full(shape, fill)
        x = x.to(torch.bfloat16).to(dtype)
        out.append(x.transpose(-3, -2) if layout == "head" else x)
    return out


def tables(B, max_pages, num_pages, g):
    """Page tables of distinct pages in no order."""
    return torch.randperm(num_pages, generator=g)[: B * max_pages].view(B, max_pages).to(torch.int32)


def at(pages, b, slot, page):
    return int(pages[b, slot // page]), slot % page


def to_cuda(x):
    """The tensor on the GPU with its strides kept."""
    if x is None:
        return None
    base = x.as_strided((x.untyped_storage().nbytes() // x.element_size(),), (1,), 0)
    raw = base.view(torch.uint8) if x.dtype == F8 else base
    dev = raw.cuda()
    dev = dev.view(F8) if x.dtype == F8 else dev
    return dev.as_strided(x.shape, x.stride(), x.storage_offset())


def attention(q, k_cache, v_cache, pages, ctx, tb, mask, scale, k_scale=None, v_scale=None):
    """(out, bound): attention of every new token in float64, and the elementwise error bound of a result
    with fp32 scores and sums, weights rounded to bf16 or fp16 and a bf16 output.

    Per element, with w the weights summing to 1 and A = sum w |v|: the output rounds by 2^-8 |o|; a
    weight's rounding is 2^-8 of it at most (bf16; fp16's is smaller, and its underflow adds 2^-24 of
    the largest weight per slot), so 2^-8 A; a score's fp32 sum of D products is off by at most
    (D + 2) 2^-24 scale sum |q k|, twice that in a normalised weight; exp2, its argument's scaling
    (2^-22 |score| in an absolute error) and the sums add 2^-18 A."""
    B, T, Hq, D = q.shape
    page, H = k_cache.shape[1], k_cache.shape[2]
    G = Hq // H
    out = torch.zeros(q.shape, dtype=torch.float64)
    bound = torch.zeros(q.shape, dtype=torch.float64)
    for b in range(B):
        for t in range(tb[b]):
            rule = (1 << (t + 1)) - 1 if mask is None else int(mask[b, t])
            slots = [s for s in range(ctx[b] + tb[b]) if s < ctx[b] or (rule >> (s - ctx[b])) & 1]
            if not slots:
                continue
            where = [at(pages, b, s, page) for s in slots]
            p = torch.tensor([w[0] for w in where])
            r = torch.tensor([w[1] for w in where])
            raw = [(c.contiguous().view(torch.uint8) if c.dtype == F8 else c)[p, r] for c in (k_cache, v_cache)]
            k, v = [(x.view(F8) if k_cache.dtype == F8 else x).to(torch.float64).transpose(0, 1) for x in raw]
            if k_scale is not None:
                k = k * k_scale.double()[:, None, None]
            if v_scale is not None:
                v = v * v_scale.double()[:, None, None]
            qq = q[b, t].double().view(H, G, D)
            z = qq @ k.transpose(1, 2) * scale
            size = qq.abs() @ k.abs().transpose(1, 2) * abs(scale)
            w = torch.softmax(z, -1)
            o = w @ v
            rel = 2 * ((D + 2) * U_F32 * size + 2.0 ** -22 * z.abs()).amax(-1, keepdim=True) + 2.0 ** -18
            small = len(slots) * 2.0 ** -24 * w.amax(-1, keepdim=True) * v.abs().amax(1)[:, None]
            out[b, t] = o.reshape(Hq, D)
            bound[b, t] = (U_BF16 * 1.01 * o.abs() + (U_BF16 + rel) * (w @ v.abs()) + small).reshape(Hq, D)
    return out, bound


def rotate(x, cos, sin, interleaved):
    """(rotated, bound) of [..., D] in float64: fp32 products and their sum are off by 2^-22 (|x| + |y|)."""
    r = 2 * len(cos)
    y, e = x.clone(), torch.zeros_like(x)
    for i in range(r // 2):
        a, c = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        y[..., a] = x[..., a] * cos[i] - x[..., c] * sin[i]
        y[..., c] = x[..., c] * cos[i] + x[..., a] * sin[i]
        e[..., a] = e[..., c] = 2.0 ** -22 * (x[..., a].abs() + x[..., c].abs())
    return y, e


def logits(z, rules, tb):
    """(out, bound) of process_logits in float64 (out is NaN where nothing is written); numpy arrays."""
    B, T, V = z.shape
    out = np.full(z.shape, np.nan)
    bound = np.zeros(z.shape)
    get = lambda name: rules.get(name)  # noqa: E731
    for b in range(B):
        count, prompt = np.zeros(V), np.zeros(V, bool)
        if get("history") is not None:
            held = min(max(int(rules["history_len"][b]), 0), rules["history"].shape[1])
            start = int(rules["prompt_len"][b]) if get("prompt_len") is not None else 0
            for i in range(held):
                v = int(rules["history"][b, i])
                if 0 <= v < V:
                    if i < start:
                        prompt[v] = True
                    else:
                        count[v] += 1
        bias = np.zeros(V)
        if get("bias_ids") is not None:
            for i, v in enumerate(rules["bias_ids"][b]):
                if 0 <= v < V:
                    bias[v] = rules["bias"][b, i]
        rep, pre, fre = (float(rules[n][b]) if get(n) is not None else d
                         for n, d in (("repetition", 1.0), ("presence", 0.0), ("frequency", 0.0)))
        for t in range(tb[b]):
            if t > 0 and get("draft") is not None and 0 <= rules["draft"][b, t - 1] < V:
                count[rules["draft"][b, t - 1]] += 1
            x = z[b, t].astype(np.float64)
            with np.errstate(invalid="ignore"):
                seen = prompt | (count > 0)
                y = np.where(seen, np.where(x > 0, x / rep, x * rep), x)
                size = np.abs(y) + abs(fre) * count + abs(pre) * (count > 0) + np.abs(bias)
                y = y - fre * count - pre * (count > 0) + bias
            if get("mask") is not None:
                bits = (rules["mask"][b, t].astype(np.int64)[np.arange(V) // 32] >> (np.arange(V) % 32)) & 1
                y[bits == 0] = -math.inf
            out[b, t] = y
            bound[b, t] = np.where(np.isfinite(size), 6 * U_F32 * size, 0.0)
    return out, bound
