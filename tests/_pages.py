"""Inputs and 64-bit references of the tests of page scales and eviction: one entry, page and row at a time, on the CPU."""
from __future__ import annotations

import math

import torch

import _decode as R

F8_MAX = 448.0


def need(most: float) -> float:
    """The smallest power of two s in 2^-24 .. 2^24 with most <= 448 s."""
    k = -24
    while k < 24 and most > F8_MAX * 2.0 ** k:
        k += 1
    return 2.0 ** k


def codes_of(x):
    """float64 values as E4M3 codes' values: nearest, ties to even, cut to +-448, NaN kept (through float32: the
    inputs here have few enough bits for that to be exact, or are compared with a tolerance)."""
    return x.float().clamp(-F8_MAX, F8_MAX).to(R.F8)


def counts(s: float) -> bool:
    return 2.0 ** -24 <= s <= 2.0 ** 24


def pool(num_pages, page, H, D, layout, g, layers=None, spread=3):
    """(k, v, k_scale, v_scale) on the CPU: codes that fill their range, scales powers of two up to 2^spread apart."""
    k, v = R.pool(num_pages, page, H, D, R.F8, layout, g, layers)
    for c in (k, v):
        x = torch.randn(c.shape, generator=g) * 100
        c.view(torch.uint8).copy_(x.clamp(-F8_MAX, F8_MAX).to(R.F8).view(torch.uint8))
    lead = () if layers is None else (layers,)
    scale = lambda: 2.0 ** torch.randint(-8, -7 + spread, lead + (num_pages, H), generator=g).float()  # noqa: E731
    return k, v, scale(), scale()


def values(cache, scale):
    """The entries [.., pages, page, heads, D] in float64."""
    return cache.contiguous().view(torch.uint8).view(R.F8).double() * scale.double()[..., :, None, :, None]


def put(cache, scale, page, head, rows, x, stays):
    """Entries x [n, D] (float64) go to `rows` of one page and head; `stays`: rows that keep what they hold (None: the page
    starts anew).  Changes cache and scale in place."""
    raw = cache.view(torch.uint8)
    fine = x.abs()[torch.isfinite(x)]
    new, old = need(float(fine.max()) if fine.numel() else 0.0), float(scale[page, head])
    if stays is not None and counts(old):
        if new > old:
            for r in stays:
                raw[page, r, head] = codes_of(raw[page, r, head].view(R.F8).double() * (old / new)).view(torch.uint8)
        new = max(old, new)
    for r, e in zip(rows, x):
        raw[page, r, head] = codes_of(e / new).view(torch.uint8)
    scale[page, head] = new


def moved(cache, scale, pages, pairs, head, end, page):
    """One (request, head) of a keep or move, in place: pairs of (source, target) slots; slots < end keep their values."""
    raw = cache.view(torch.uint8)
    before, was = raw.clone(), scale.clone()
    at = lambda s: (int(pages[s // page]), s % page)  # noqa: E731
    for p in sorted({t // page for _, t in pairs}):
        mine = [(s, t) for s, t in pairs if t // page == p]
        x = torch.stack([before[at(s)[0], at(s)[1], head].view(R.F8).double() * float(was[at(s)[0], head]) for s, _ in mine])
        taken = {t for _, t in mine}
        stays = [n % page for n in range(p * page, min((p + 1) * page, end)) if n not in taken]
        put(cache, scale, at(mine[0][1])[0], head, [t % page for _, t in mine], x, stays)


def scores(q, k, pages, ctx, tb, mask, scale, f8):
    """Per (b, t): (slots, z [H, G, n], error bound of z).  k: values [pages, page, heads, D] in float64.

    A score is a sum of D products in fp32: (D + 2) 2^-24 of the sum of their magnitudes, and a conversion to log2 units and
    back (2^-22 of it).  Over an E4M3 cache elements of q below 2^-9 of the row's largest are off by 2^-17 of that."""
    B, T, Hq, D = q.shape
    page, H = k.shape[1:3]
    for b in range(B):
        for t in range(tb[b]):
            rule = (1 << (t + 1)) - 1 if mask is None else int(mask[b, t])
            slots = [s for s in range(ctx[b] + tb[b]) if s < ctx[b] or (rule >> (s - ctx[b])) & 1]
            if not slots:
                continue
            n = torch.tensor(slots)
            kk = k[pages[b].long()[n // page], n % page].transpose(0, 1)  # [H, n, D]
            qq = q[b, t].double().view(H, Hq // H, D)
            z = qq @ kk.transpose(1, 2) * scale
            size = qq.abs() @ kk.abs().transpose(1, 2) * abs(scale)
            e = (D + 2) * R.U_F32 * size + 2.0 ** -22 * z.abs()
            if f8:
                e = e + 2.0 ** -17 * qq.abs().amax(-1)[..., None] * kk.abs().sum(-1)[:, None] * abs(scale)
            yield b, t, n, z, e


def lse(q, k, pages, ctx, tb, mask, scale, f8):
    """(lse [B, T, Hq], bound)."""
    B, T, Hq, _ = q.shape
    out = torch.full((B, T, Hq), -math.inf, dtype=torch.float64)
    bound = torch.zeros_like(out)
    for b, t, _, z, e in scores(q, k, pages, ctx, tb, mask, scale, f8):
        total = torch.logsumexp(z, -1)
        out[b, t] = total.view(-1)
        bound[b, t] = (e.amax(-1) + 2.0 ** -18 + 2.0 ** -21 * total.abs()).view(-1)
    return out, bound


def weigh(q, k, pages, ctx, tb, mask, scale, given, weight, position, positions, f8):
    """(weight, position, bound) after kv_weigh: weight [pages, heads, page] float64."""
    B, T, Hq, _ = q.shape
    page, H = k.shape[1:3]
    weight, position = weight.double().clone(), position.clone()
    bound = torch.zeros_like(weight)
    for b in range(B):
        for t in range(tb[b]):
            s = ctx[b] + t
            weight[pages[b, s // page], :, s % page] = 0.0
            position[pages[b, s // page], :, s % page] = s if positions is None else positions[b, t]
    for b, t, n, z, e in scores(q, k, pages, ctx, tb, mask, scale, f8):
        total = given[b, t].double().view(H, -1, 1)
        w = torch.where(torch.isinf(total), 0.0, torch.exp(z - torch.where(torch.isinf(total), 0.0, total)))
        off = w * (e + 2.0 ** -22 * (z.abs() + torch.where(torch.isinf(total), 0.0, total).abs()) + 2.0 ** -19)
        weight[pages[b].long()[n // page], :, n % page] += w.sum(1).T
        bound[pages[b].long()[n // page], :, n % page] += off.sum(1).T
    rows = 2 + T * Hq // H
    return weight, position, bound + rows * R.U_F32 * weight.abs()


def select(weight, position, pages, ctx, budget, seen, first, recent):
    """Per request and head: (sources, targets), and the new lengths.  weight [pages, heads, page]."""
    page, H = weight.shape[2], weight.shape[1]
    out, length = [], []
    for b, n in enumerate(ctx):
        n = max(n, 0)
        m = min(n, max(budget[b], 0))
        length.append(m)
        row = []
        for h in range(H):
            key = []
            for s in range(n):
                p = int(pages[b, s // page])
                w = -math.inf
                if 0 <= p < weight.shape[0]:
                    w = float(weight[p, h, s % page])
                    w = -math.inf if math.isnan(w) else w
                    if position is not None:
                        at = int(position[p, h, s % page])
                        if at < first or (recent > 0 and at >= (seen[b] if seen is not None else n) - recent):
                            w = math.inf
                key.append(w)
            kept = set(sorted(range(n), key=lambda s: (-key[s], s))[:m])
            row.append(([s for s in range(m, n) if s in kept], [s for s in range(m) if s not in kept]))
        out.append(row)
    return out, length
