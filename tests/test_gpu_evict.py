"""kv_weigh, kv_select and kv_move against the definitions in 64 bits, and the whole of them as a decode loop uses them."""
import math

import pytest
import torch

import _decode as R
import _pages as P

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------
# weigh
# ------------------------------------------------------------------------------------------------
def build(kind, B, T, Hq, H, D, page, ctx, layout="slot", seed=1, mask=None, tb=None):
    g = torch.Generator().manual_seed(seed)
    max_pages = -(-(max(ctx) + T) // page) + 1
    num_pages = B * max_pages + 2
    tb = [T] * B if tb is None else tb
    pages = R.tables(B, max_pages, num_pages, g)
    ks = None
    if kind == "pages":
        k, _, ks, _ = P.pool(num_pages, page, H, D, layout, g)
    else:
        k, _ = R.pool(num_pages, page, H, D, BF if kind == "bf16" else R.F8, layout, g)
        ks = torch.rand(H, generator=g) + 0.5 if kind == "e4m3" else None
    used = torch.zeros((num_pages, page), dtype=torch.bool)
    for b in range(B):
        for s in range(ctx[b] + tb[b]):
            used[R.at(pages, b, s, page)] = True
        pages[b, -(-(ctx[b] + tb[b]) // page):] = 2 ** 30 + b
    raw = k if kind == "bf16" else k.view(torch.uint8)
    raw[~used] = float("nan") if kind == "bf16" else 0x7F
    if kind == "pages":
        ks[~used.any(1)] = math.nan
        values = P.values(k, ks)
    else:
        values = k.double() if kind == "bf16" else k.contiguous().view(torch.uint8).view(R.F8).double() * ks.double()[:, None]
    values = torch.nan_to_num(values)
    q = (torch.randn((B, T, Hq, D), generator=g) * 1.5).to(BF)
    lse, _ = P.lse(q, values, pages, ctx, tb, mask, D ** -0.5, False)
    weight = torch.rand((num_pages, H, page), generator=g)
    weight[~used[:, None].expand(weight.shape)] = math.nan
    for b in range(B):  # what new slots held before has no part
        for t in range(tb[b]):
            p, r = R.at(pages, b, ctx[b] + t, page)
            weight[p, :, r] = math.nan
    return dict(q=q, k=k, ks=ks, values=values, pages=pages, ctx=ctx, tb=tb, mask=mask, lse=lse.float(), weight=weight,
                position=torch.randint(0, 99, weight.shape, generator=g).to(torch.int32), scale=D ** -0.5, f8=kind != "bf16")


def weigh(d, positions=None, with_position=True, **kw):
    import speculative_decoding_rejection_verify_gb300 as sv
    w, p = d["weight"].cuda(), d["position"].cuda()
    sv.kv_weigh(d["q"].cuda(), R.to_cuda(d["k"]), d["pages"].cuda(), i32(d["ctx"]), d["lse"].cuda(), w, p if with_position else None,
                t_per_row=i32(d["tb"]), mask=None if d["mask"] is None else d["mask"].cuda(), scale=d["scale"],
                positions=None if positions is None else positions.cuda(), k_scale=R.to_cuda(d["ks"]), **kw)
    torch.cuda.synchronize()
    return w.cpu(), p.cpu()


def check(d, positions=None, **kw):
    w, p = weigh(d, positions, **kw)
    want, want_p, bound = P.weigh(d["q"], d["values"], d["pages"], d["ctx"], d["tb"], d["mask"], d["scale"], d["lse"], d["weight"],
                                  d["position"], positions, d["f8"])
    assert torch.equal(p, want_p)
    assert torch.equal(torch.isnan(w), torch.isnan(want))
    off = torch.nan_to_num((w.double() - want).abs())
    assert (off <= torch.nan_to_num(bound)).all(), f"over the bound by {(off - bound).nan_to_num().max():.3g}"
    return w


KINDS = ["bf16", "e4m3", "pages"]


@pytest.mark.parametrize("T,Hq,H,D", [(1, 1, 1, 64), (1, 8, 8, 128), (1, 8, 2, 64), (5, 8, 2, 128), (6, 7, 1, 128),
                                      (3, 15, 5, 64), (17, 8, 1, 128), (9, 12, 1, 64), (17, 8, 2, 64), (64, 6, 2, 128),
                                      (1, 128, 1, 128), (64, 12, 2, 64), (2, 128, 1, 128)])
@pytest.mark.parametrize("kind", KINDS)
def test_weigh_head_layouts(T, Hq, H, D, kind):
    check(build(kind, 2, T, Hq, H, D, 16, [37, 300]))


@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 63, 125, 126, 127, 128, 129, 255, 256, 640])
@pytest.mark.parametrize("kind", KINDS)
def test_weigh_lengths(ctx, kind):
    check(build(kind, 1, 3, 4, 2, 128, 16, [ctx], seed=ctx))


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("layout", ["slot", "head"])
@pytest.mark.parametrize("kind", KINDS)
def test_weigh_pages_and_orders(page, layout, kind):
    check(build(kind, 3, 4, 8, 2, 128, page, [5, 130, 517], layout, seed=page))
    check(build(kind, 2, 2, 4, 2, 64, page, [1, 260], layout, seed=page))


@pytest.mark.parametrize("kind", KINDS)
def test_weigh_ragged(kind):
    ctx, tb = [0, 5, 900, 0, 64, 2000, 1, 130], [0, 3, 0, 5, 1, 5, 2, 4]
    check(build(kind, 8, 5, 8, 2, 128, 16, ctx, tb=tb))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq,H,T", [(4, 2, 9), (48, 1, 9), (64, 2, 64)])
def test_weigh_trees(kind, Hq, H, T):
    g = torch.Generator().manual_seed(Hq)
    mask = torch.randint(-2 ** 63, 2 ** 63 - 1, (3, T), generator=g, dtype=torch.int64)
    mask[0, 0] = 0
    d = build(kind, 3, T, Hq, H, 64, 16, [0, 200, 33], mask=mask)
    check(d, positions=torch.randint(0, 500, (3, T), generator=g).to(torch.int32))


@pytest.mark.parametrize("kind", KINDS)
def test_weigh_rows_without_a_part(kind):
    """Rows whose sum is infinite add nothing; without positions none are written."""
    d = build(kind, 2, 4, 8, 2, 64, 16, [50, 300])
    d["lse"][0, 2:] = math.inf
    d["lse"][1, 1, 3] = -math.inf
    w = check(d)
    again, p = weigh(d, with_position=False)
    assert torch.equal(p, d["position"]) and torch.equal(torch.nan_to_num(again), torch.nan_to_num(w))


@pytest.mark.parametrize("kind", KINDS)
def test_weigh_a_wide_table_and_pages_outside(kind):
    d = build(kind, 2, 4, 8, 2, 64, 16, [50, 300])
    w = check(d)
    wide = dict(d, pages=torch.cat([d["pages"], torch.full((2, 3000), -9, dtype=torch.int32)], 1))
    assert torch.equal(torch.nan_to_num(weigh(wide)[0]), torch.nan_to_num(w))
    gone = dict(d, pages=d["pages"].clone())
    lost = int(gone["pages"][1, 3])
    gone["pages"][1, 3] = -1
    got = weigh(gone)[0]
    assert torch.equal(torch.nan_to_num(got[lost]), torch.nan_to_num(d["weight"][lost]))
    keep = torch.arange(len(w)) != lost
    assert torch.equal(torch.nan_to_num(got[keep]), torch.nan_to_num(w[keep]))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tb", [None, [1 + i % 3 for i in range(60)]])
def test_weigh_many_short_items(kind, tb):
    """Several items of one or two tiles a block, of which each warpgroup has some and passes the others by."""
    check(build(kind, 60, 3, 16, 8, 64, 16, [(37 * i) % 300 for i in range(60)], tb=tb))


@pytest.mark.parametrize("kind", KINDS)
def test_weigh_many_rows_sums_to_the_rows(kind):
    """Every row's weights sum to 1, so a step adds as much as it has rows (2^-12: 2^-24 a weight and the bound of the scores)."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(2)
    B, T, Hq, H, D, page, n = 3, 7, 16, 4, 128, 32, 5000
    maxp = -(-(n + T) // page)
    k = torch.randn((B * maxp, page, H, D), generator=g).to(BF)
    k = k if kind == "bf16" else k.to(R.F8)
    k, ks = k.cuda(), None if kind != "pages" else torch.full((B * maxp, H), 0.5, device="cuda")
    pages = torch.arange(B * maxp, dtype=torch.int32).view(B, maxp).cuda()
    q, ctx = torch.randn((B, T, Hq, D), generator=g).to(BF).cuda(), i32([n, 17, 4000])
    lse, w = torch.zeros((B, T, Hq), device="cuda"), torch.zeros((B * maxp, H, page), device="cuda")
    sv.paged_attention(q, k, k, pages, ctx, k_scale=ks, v_scale=ks, lse=lse)
    sv.kv_weigh(q, k, pages, ctx, lse, w, k_scale=ks)
    got = w.double().view(B, maxp, H, page).sum((1, 3))
    tol = T * Hq / H * (2.0 ** -12 + (2.0 ** -8 if kind == "bf16" else 0.0))  # a bf16 cache's sums are rounded weights'
    assert ((got - T * Hq / H).abs() <= tol).all()


# ------------------------------------------------------------------------------------------------
# select
# ------------------------------------------------------------------------------------------------
def run_select(weight, position, pages, ctx, budget, seen=None, first=0, recent=0, **kw):
    import speculative_decoding_rejection_verify_gb300 as sv
    src, dst, n, m = sv.kv_select(weight.cuda(), None if position is None else position.cuda(), pages.cuda(), i32(ctx), i32(budget),
                                  seen=None if seen is None else i32(seen), first=first, recent=recent, **kw)
    torch.cuda.synchronize()
    src, dst, n = src.cpu(), dst.cpu(), n.cpu()
    layered = weight if weight.dim() == 4 else weight[None]
    for layer in range(layered.shape[0]):
        want, length = P.select(layered[layer], None if position is None else (position if weight.dim() == 3 else position[layer]), pages,
                                ctx, budget, seen, first, recent)
        assert m.tolist() == length
        pick = (lambda x: x) if weight.dim() == 3 else (lambda x: x[layer])
        for b, row in enumerate(want):
            for h, (sources, targets) in enumerate(row):
                k = len(sources)
                assert pick(n)[b, h] == k
                assert pick(src)[b, h, :k].tolist() == sources and pick(dst)[b, h, :k].tolist() == targets
    return src, dst, n, m


def record(B, H, page, slots, g, layers=None, ties=False):
    maxp = -(-slots // page)
    num = B * maxp + 2
    shape = (() if layers is None else (layers,)) + (num, H, page)
    w = torch.randint(0, 5, shape, generator=g).float() * 0.25 if ties else torch.rand(shape, generator=g) ** 8
    return w, torch.randint(0, 2 * slots, shape, generator=g).to(torch.int32), R.tables(B, maxp, num, g)


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("slots", [1, 2, 7, 31, 32, 33, 100, 1000, 1023, 1024, 1025, 2500, 9000])
def test_select_lengths(slots, ties):
    g = torch.Generator().manual_seed(slots)
    w, p, pages = record(3, 2, 16, slots, g, ties=ties)
    run_select(w, p, pages, [slots, slots // 2, max(slots - 3, 0)], [slots // 3, slots - 1, slots // 2], [slots] * 3, 2, slots // 5)


@pytest.mark.parametrize("page", [8, 64, 512, 4096])
def test_select_pages_and_layers(page):
    g = torch.Generator().manual_seed(page)
    w, p, pages = record(4, 3, page, 700, g, layers=2)
    run_select(w, p, pages, [700, 0, 350, 699], [300, 10, 350, 1], [900, 5, 800, 701], 4, 64)


def test_select_budgets_at_the_edges():
    g = torch.Generator().manual_seed(4)
    w, p, pages = record(6, 2, 16, 200, g)
    run_select(w, None, pages, [200, 200, 200, 0, 1, -5], [0, -7, 2 ** 31 - 1, 5, 1, 3])


def test_select_odd_weights():
    """Ties at every weight, -0 and +0 alike, infinities, NaN as -infinity, negative ones, more protected ones than the budget."""
    g = torch.Generator().manual_seed(9)
    w, p, pages = record(2, 4, 8, 300, g)
    odd = torch.tensor([0.0, -0.0, math.inf, -math.inf, math.nan, -1.0, 1.0, 1e-45, -1e-45, 3.4e38])
    w = odd[torch.randint(0, len(odd), w.shape, generator=g)]
    w[:, 3] = 1.0
    run_select(w, None, pages, [300, 211], [100, 3])
    run_select(w, p, pages, [300, 211], [10, 150], None, 600, 0)
    run_select(w, p, pages, [300, 211], [100, 30], [500, 211], 0, 100)
    run_select(w, p, pages, [300, 211], [100, 30], [2 ** 31 - 1, 5], 0, 2 ** 31 - 1)


def test_select_pages_outside_the_pool_go_first():
    g = torch.Generator().manual_seed(5)
    w, p, pages = record(1, 2, 8, 100, g)
    pages[0, 2], pages[0, 5] = -1, 2 ** 30
    run_select(w + 1.0, p, pages, [100], [60], [100], 0, 30)


def test_select_long():
    g = torch.Generator().manual_seed(6)
    w, p, pages = record(1, 1, 64, 70001, g, ties=True)
    run_select(w, p, pages, [70001], [20000], [140000], 4, 3000)
    w, p, pages = record(1, 2, 64, 250000, g)
    run_select(w, p, pages, [250000], [249990], [500000], 0, 100)


def test_select_leaves_the_rest_of_the_lists():
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(7)
    w, p, pages = record(2, 2, 8, 64, g)
    new = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
    out = new(2, 2, 40), new(2, 2, 40), new(2, 2), new(2)
    got = sv.kv_select(w.cuda(), p.cuda(), pages.cuda(), i32([64, 20]), i32([30, 25]), out=out)
    assert all(a is b for a, b in zip(got, out))
    for lists in out[:2]:
        for b in range(2):
            for h in range(2):
                k = int(out[2][b, h])
                assert (lists[b, h, k:] == -9).all() and (lists[b, h, :k] >= 0).all()


# ------------------------------------------------------------------------------------------------
# move
# ------------------------------------------------------------------------------------------------
def run_move(kind, B, H, D, page, ctx, budget, layout="slot", layers=None, seed=1, far=False):
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(seed)
    slots = max(ctx)
    w, pos, pages = record(B, H, page, slots, g, layers)
    num = w.shape[-3]
    ks = vs = None
    if kind == "pages":
        k, v, ks, vs = P.pool(num, page, H, D, layout, g, layers)
        if far:
            ks, vs = (2.0 ** torch.randint(-20, 20, x.shape, generator=g).float() for x in (ks, vs))
    else:
        k, v = R.pool(num, page, H, D, BF if kind == "bf16" else R.F8, layout, g, layers)
    dev = [R.to_cuda(x) for x in (k, v)] + [None if x is None else x.cuda() for x in (ks, vs)] + [w.cuda(), pos.cuda()]
    src, dst, n, m = sv.kv_select(dev[4], None, pages.cuda(), i32(ctx), i32(budget))
    sv.kv_move(dev[0], dev[1], pages.cuda(), m, src, dst, n, k_scale=dev[2], v_scale=dev[3], weight=dev[4], position=dev[5])
    torch.cuda.synchronize()
    src, dst, n, m = (x.cpu() for x in (src, dst, n, m))
    k, v = k.contiguous(), v.contiguous()
    raw = [x if kind == "bf16" else x.view(torch.uint8) for x in (k, v)]
    for layer in range(layers or 1):
        side = lambda x: x if layers is None else x[layer]  # noqa: E731
        for b in range(B):
            for h in range(H):
                c = int(side(n)[b, h])
                pairs = list(zip(side(src)[b, h, :c].tolist(), side(dst)[b, h, :c].tolist()))
                at = lambda s: (int(pages[b, s // page]), s % page)  # noqa: E731
                if kind == "pages":
                    if pairs:
                        P.moved(side(k), side(ks), pages[b], pairs, h, int(m[b]), page)
                        P.moved(side(v), side(vs), pages[b], pairs, h, int(m[b]), page)
                for s, t in pairs:
                    if kind != "pages":
                        for x in raw:
                            side(x)[at(t)[0], at(t)[1], h] = side(x)[at(s)[0], at(s)[1], h]
                    for x in (w, pos):
                        side(x)[at(t)[0], h, at(t)[1]] = side(x)[at(s)[0], h, at(s)[1]]
    for got, want in zip(dev, (k, v, ks, vs, w, pos)):
        if got is not None:
            got = got.cpu().contiguous()
            if got.dtype == R.F8:
                got, want = got.view(torch.uint8), want.view(torch.uint8)
            assert torch.equal(got, want), int((got != want).sum())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("layout", ["slot", "head"])
@pytest.mark.parametrize("page,D", [(8, 64), (16, 128), (64, 64), (256, 128), (2048, 64)])
def test_move(kind, layout, page, D):
    run_move(kind, 3, 2, D, page, [300, 77, 211], [100, 77, 205], layout, seed=page)


@pytest.mark.parametrize("kind", KINDS)
def test_move_layers(kind):
    run_move(kind, 2, 3, 64, 16, [200, 130], [77, 64], layers=3)


@pytest.mark.parametrize("budget", [1, 7, 8, 9, 63, 64, 65, 127, 128, 199])
def test_move_ends_within_and_between_pages(budget):
    run_move("pages", 1, 2, 64, 8, [200], [budget], seed=budget, far=True)
    run_move("pages", 1, 1, 128, 64, [200], [budget], seed=budget, far=True)


def test_move_many():
    run_move("pages", 1, 1, 64, 32, [9000], [4000], far=True)
    run_move("bf16", 1, 1, 64, 512, [9000], [4500])


def test_move_leaves_out_what_lies_outside():
    """Targets behind the context, sources before its end or behind the table, pages outside the pool, counts out of range."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(3)
    w, pos, pages = record(1, 1, 8, 64, g)
    for kind in KINDS:
        k, v = R.pool(w.shape[0], 8, 1, 64, BF if kind == "bf16" else R.F8, "slot", g)
        s = torch.ones((w.shape[0], 1), device="cuda") if kind == "pages" else None
        dev, t = [x.cuda() for x in (k, v)], pages.clone()
        t[0, 6] = -1
        src, dst = i32([[[48, 3, 64, 2 ** 31 - 1, 40]]]), i32([[[1, 2, 3, 4, 20]]])
        sv.kv_move(*dev, t.cuda(), i32([20]), src, dst, i32([[9]]), k_scale=s, v_scale=s)
        sv.kv_move(*dev, t.cuda(), i32([20]), src, dst, i32([[-1]]), k_scale=s, v_scale=s)
        torch.cuda.synchronize()
        for got, want in zip(dev, (k, v)):
            assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))


# ------------------------------------------------------------------------------------------------
# all of it together
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind", KINDS)
def test_a_decode_loop_within_a_budget(kind):
    """Steps of append, attend and weigh, with an eviction when the cache is over its budget.  Each operator's result is compared with its
    definition on what was in memory before it; at the end every head's recorded positions are distinct, hold the protected ones,
    and every entry is the one that was appended at its position."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(8)
    B, T, Hq, H, D, page, budget, first, recent = 2, 4, 8, 2, 64, 16, 40, 2, 12
    maxp = 5
    num = B * maxp + 1
    pages = torch.randperm(num, generator=g)[: B * maxp].view(B, maxp).to(torch.int32)
    dt = BF if kind == "bf16" else R.F8
    k, v = (torch.zeros((num, page, H, D), dtype=BF).to(dt).cuda() for _ in range(2))
    scales = {n: torch.ones((num, H), device="cuda") for n in ("k_scale", "v_scale")} if kind == "pages" else {}
    key = {"k_scale": scales["k_scale"]} if scales else {}
    weight, position = torch.zeros((num, H, page), device="cuda"), torch.zeros((num, H, page), dtype=torch.int32, device="cuda")
    ctx, seen, dev_pages = i32([0, 0]), i32([0, 0]), pages.cuda()
    written = torch.zeros((B, 200, 2, H, D))
    for step in range(30):
        qkv = torch.randn((B, T, Hq + 2 * H, D), generator=g).to(BF)
        tb = [T, 1 + step % T]
        q, kk, vv = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:]
        at = (seen[:, None] + torch.arange(T, dtype=torch.int32, device="cuda")).contiguous()
        for b in range(B):
            for t in range(tb[b]):
                written[b, int(seen[b]) + t, 0], written[b, int(seen[b]) + t, 1] = kk[b, t].float(), vv[b, t].float()
        qr = sv.kv_append(q.cuda(), kk.cuda(), vv.cuda(), k, v, dev_pages, ctx, t_per_row=i32(tb), **scales)
        lse = torch.zeros((B, T, Hq), device="cuda")
        out = sv.paged_attention(qr, k, v, dev_pages, ctx, i32(tb), lse=lse, **scales)
        before = weight.cpu()
        sv.kv_weigh(qr, k, dev_pages, ctx, lse, weight, position, t_per_row=i32(tb), positions=at, **key)
        torch.cuda.synchronize()
        deq = [P.values(x.cpu(), s.cpu()) if scales else x.cpu().to(torch.float64) for x, s in zip((k, v), scales.values() or (0, 0))]
        n = ctx.tolist()
        want, bound = R.attention(q, *deq, pages, n, tb, None, D ** -0.5)
        assert ((out.cpu().double() - want).abs() <= bound).all()
        want, _, bound = P.weigh(q, deq[0], pages, n, tb, None, D ** -0.5, lse.cpu(), before, position.cpu(), at.cpu(), kind != "bf16")
        assert ((weight.cpu().double() - want).abs() <= bound).all()
        ctx, seen = ctx + i32(tb), seen + i32(tb)
        if int(ctx.max()) > budget + 16:
            src, dst, moves, ctx = sv.kv_select(weight, position, dev_pages, ctx, i32([budget] * B), seen=seen, first=first, recent=recent)
            sv.kv_move(k, v, dev_pages, ctx, src, dst, moves, weight=weight, position=position, **scales)
    torch.cuda.synchronize()
    deq = [P.values(x.cpu(), s.cpu()) if scales else x.cpu().to(torch.float64) for x, s in zip((k, v), scales.values() or (0, 0))]
    for b in range(B):
        n, total = int(ctx[b]), int(seen[b])
        assert n < total
        slots = torch.arange(n)
        p, r = pages[b].long()[slots // page], slots % page
        for h in range(H):
            held = position.cpu()[p, h, r]
            assert len(set(held.tolist())) == n
            assert set(range(first)) <= set(held.tolist()) and set(range(total - recent, total)) <= set(held.tolist())
            for x, entry in zip((0, 1), deq):
                want = written[b, held.long(), x, h].double()
                # E4M3: half a step of 2^-4 each time an entry is coded (when its page's scale grows it changes only where it becomes
                # subnormal: 2^-10 of the scale each time, and scales grow a few powers of two here)
                tol = 0.0 if kind == "bf16" else 2.0 ** -4 * want.abs() + (2.0 ** -10 if kind == "e4m3" else 8 * 2.0 ** -10 * 2.0 ** -6)
                assert ((entry[p, r, h] - want).abs() <= tol).all()


def test_eviction_captured_and_replayed():
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(12)
    w, pos, pages = record(2, 2, 16, 200, g)
    k, v, ks, vs = P.pool(w.shape[0], 16, 2, 64, "slot", g)
    dev = [R.to_cuda(x) for x in (k, v)] + [x.cuda() for x in (ks, vs, w, pos)]
    t, ctx, budget = pages.cuda(), i32([200, 150]), i32([64, 100])

    def evict(x):
        src, dst, n, m = sv.kv_select(x[4], x[5], t, ctx, budget, first=2, recent=20)
        sv.kv_move(x[0], x[1], t, m, src, dst, n, k_scale=x[2], v_scale=x[3], weight=x[4], position=x[5])
        return m

    first = [x.clone() for x in dev]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        evict([x.clone() for x in dev])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        evict(dev)
    for seed in range(2):
        for x, y in zip(dev, first):
            x.view(torch.uint8).copy_(y.view(torch.uint8))
        dev[4].copy_(torch.rand(w.shape, generator=g))
        twin = [x.clone() for x in dev]
        graph.replay()
        m = evict(twin)
        torch.cuda.synchronize()
        assert m.tolist() == [64, 100]
        for x, y in zip(dev, twin):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("kind", KINDS)
def test_weigh_waits_that_give_up_leave_nan(kind):
    import speculative_decoding_rejection_verify_gb300 as sv
    d = build(kind, 3, 4, 8, 2, 128, 16, [700, 1900, 300])
    want = weigh(d)[0]
    sv.set_test_hooks(2)
    try:
        got = weigh(d)[0]
    finally:
        sv.set_test_hooks(0)
    same = torch.nan_to_num(got, nan=-1.0) == torch.nan_to_num(want, nan=-1.0)
    assert (same | torch.isnan(got)).all() and (torch.isnan(got) & ~torch.isnan(want)).any()
    assert torch.equal(torch.nan_to_num(weigh(d)[0]), torch.nan_to_num(want))


@pytest.mark.parametrize("kind", KINDS)
def test_weigh_queries_of_a_projection(kind):
    """q with its heads between others' and its tokens in front of its requests."""
    d = build(kind, 3, 4, 8, 2, 64, 16, [5, 130, 60])
    wide = torch.full((4, 3, 14, 64), float("nan"), dtype=BF).transpose(0, 1)
    wide[:, :, 3:11] = d["q"]
    q = wide.transpose(0, 1).contiguous().cuda().transpose(0, 1)[:, :, 3:11]
    import speculative_decoding_rejection_verify_gb300 as sv
    w, p = d["weight"].cuda(), d["position"].cuda()
    sv.kv_weigh(q, R.to_cuda(d["k"]), d["pages"].cuda(), i32(d["ctx"]), d["lse"].cuda(), w, p, scale=d["scale"], k_scale=R.to_cuda(d["ks"]))
    want, want_p = weigh(d)
    assert torch.equal(torch.nan_to_num(w.cpu()), torch.nan_to_num(want)) and torch.equal(p.cpu(), want_p)


def test_eviction_on_another_stream():
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(5)
    w, pos, pages = record(2, 2, 16, 300, g)
    stream = torch.cuda.Stream()
    w, pos, t = w.cuda(), pos.cuda(), pages.cuda()
    k, v = (torch.randn((w.shape[0], 16, 2, 64), device="cuda").to(BF) for _ in range(2))
    results = []
    for s in (None, stream):
        x = [y.clone() for y in (k, v, w, pos)]
        stream.wait_stream(torch.cuda.current_stream())
        src, dst, n, m = sv.kv_select(x[2], x[3], t, i32([300, 222]), i32([100, 90]), recent=30, stream=s)
        sv.kv_move(x[0], x[1], t, m, src, dst, n, weight=x[2], position=x[3], stream=s)
        torch.cuda.synchronize()
        results.append(x)
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_empty_batches_and_tables():
    """No request, no token, no page: nothing is written, and the lists are empty."""
    import speculative_decoding_rejection_verify_gb300 as sv
    k = torch.zeros((3, 16, 2, 64), dtype=BF, device="cuda")
    w, pos = torch.ones((3, 2, 16), device="cuda"), torch.zeros((3, 2, 16), dtype=torch.int32, device="cuda")
    none = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    q = torch.zeros((0, 1, 4, 64), dtype=BF, device="cuda")
    sv.kv_weigh(q, k, none, i32([]).int(), torch.zeros((0, 1, 4), device="cuda"), w, pos)
    out = sv.kv_select(w, pos, none, i32([]).int(), i32([]).int())
    assert [tuple(x.shape) for x in out] == [(0, 2, 16), (0, 2, 16), (0, 2), (0,)]
    sv.kv_move(k, k, none, out[3], *out[:3])
    tables = torch.zeros((2, 0), dtype=torch.int32, device="cuda")
    out = sv.kv_select(w, pos, tables, i32([5, 0]), i32([3, 3]))
    assert out[2].tolist() == [[0, 0], [0, 0]] and out[3].tolist() == [0, 0]
    sv.kv_move(k, k, tables, out[3], *out[:3])
    q = torch.zeros((2, 1, 4, 64), dtype=BF, device="cuda")
    sv.kv_weigh(q, k, tables, i32([5, 0]), torch.zeros((2, 1, 4), device="cuda"), w, pos)
    torch.cuda.synchronize()
    assert (w == 1).all() and (k == 0).all()
