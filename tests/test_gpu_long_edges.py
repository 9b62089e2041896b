"""Long contexts where calls can go wrong: sums of attention whose waits gave up, lists and lengths in unusual places, queries with
large channels, and weights of drafts that were rejected."""
import math

import pytest
import torch

import _decode as R
import _pages as P

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
KINDS = ["bf16", "e4m3", "pages"]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cache(kind, num_pages, page, H, D, g, layout="slot"):
    """(k, v, scales as keyword arguments, values of k and v in float64)."""
    if kind == "pages":
        k, v, ks, vs = P.pool(num_pages, page, H, D, layout, g)
        return k, v, dict(k_scale=ks.cuda(), v_scale=vs.cuda()), P.values(k, ks), P.values(v, vs)
    k, v = R.pool(num_pages, page, H, D, BF if kind == "bf16" else R.F8, layout, g)
    if kind == "bf16":
        return k, v, {}, k.double(), v.double()
    ks, vs = (torch.rand(H, generator=g) + 0.5 for _ in range(2))
    deq = [x.contiguous().view(torch.uint8).view(R.F8).double() * s.double()[:, None] for x, s in ((k, ks), (v, vs))]
    return k, v, dict(k_scale=ks.cuda(), v_scale=vs.cuda()), *deq


# ------------------------------------------------------------------------------------------------
# the attention's sums
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("ctx", [[300, 500, 100], [700, 1900, 300]])
@pytest.mark.parametrize("Hq", [8, 40])
def test_sums_where_a_wait_gave_up_are_nan(kind, ctx, Hq):
    """Of items that one block takes whole (the narrow table) and of those that are cut and joined: what is not as it should be
    is NaN, sums as well as rows."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(4)
    B, T, H, D, page = 3, 4, 2, 128, 16
    maxp = -(-(max(ctx) + T) // page)
    k, v, scales, *_ = cache(kind, B * maxp, page, H, D, g)
    q, pages = torch.randn((B, T, Hq, D), generator=g).to(BF).cuda(), R.tables(B, maxp, B * maxp, g).cuda()
    k, v = R.to_cuda(k), R.to_cuda(v)

    def call():
        lse = torch.full((B, T, Hq), 7.0, device="cuda")
        out = sv.paged_attention(q, k, v, pages, i32(ctx), lse=lse, **scales)
        torch.cuda.synchronize()
        return out, lse

    want, sums = call()
    sv.set_test_hooks(2)
    try:
        out, lse = call()
    finally:
        sv.set_test_hooks(0)
    assert torch.isnan(out).any() and torch.isnan(lse).any()
    assert (torch.isnan(out) | (out == want)).all() and (torch.isnan(lse) | (lse == sums)).all()
    again, sums2 = call()
    assert torch.equal(again, want) and torch.equal(sums2, sums)


@pytest.mark.parametrize("Hq,D", [(2, 64), (8, 128), (40, 128), (60, 64), (84, 128)])
@pytest.mark.parametrize("ctx", [[0, 40, 700], [1, 1900, 300]])
@pytest.mark.parametrize("rising", [False, True])
def test_sums_over_bf16_are_of_weights_as_they_are(Hq, D, ctx, rising):
    """fp32's bound, without the 2^-8 of weights that are rounded to bf16; the output stays what it is without sums.  `rising`: keys
    that grow along the context, so that the maximum in use is passed again and again, by little and by more than 2^100."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(Hq)
    B, T, H, page = 3, 3, 2, 16
    maxp = -(-(max(ctx) + T) // page)
    k, v, _, kv, _ = cache("bf16", B * maxp, page, H, D, g)
    pages = R.tables(B, maxp, B * maxp, g)
    if rising:
        k *= (torch.arange(B * maxp) % 7).to(BF)[:, None, None, None]
        for b in range(B):
            k[pages[b, -4:].long()] *= 16
        kv = k.double()
    q = torch.randn((B, T, Hq, D), generator=g).to(BF)
    args = (q.cuda(), R.to_cuda(k), R.to_cuda(v), pages.cuda(), i32(ctx))
    lse = torch.zeros((B, T, Hq), device="cuda")
    out = sv.paged_attention(*args, lse=lse)
    assert torch.equal(out, sv.paged_attention(*args))
    want, bound = P.lse(q, kv, pages, ctx, [T] * B, None, D ** -0.5, False)
    off = (lse.cpu().double() - want).abs()
    assert (off <= bound).all(), f"over the bound by {(off - bound).max():.3g}"


@pytest.mark.parametrize("kind", KINDS)
def test_attention_then_weigh_adds_one_for_every_row(kind):
    """Every row's weights sum to 1: 2^-12 for the bound of the scores, for a bf16 cache too."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(3)
    B, T, Hq, H, D, page, ctx = 3, 7, 16, 4, 128, 32, [5000, 17, 4000]
    maxp = -(-(max(ctx) + T) // page)
    k, v, scales, *_ = cache(kind, B * maxp, page, H, D, g)
    if kind == "pages":
        scales["k_scale"].fill_(2.0 ** -7)
    q, k, pages = torch.randn((B, T, Hq, D), generator=g).to(BF).cuda(), k.cuda(), torch.arange(B * maxp, dtype=torch.int32).view(B, maxp).cuda()
    lse, w = torch.zeros((B, T, Hq), device="cuda"), torch.zeros((B * maxp, H, page), device="cuda")
    sv.paged_attention(q, k, v.cuda(), pages, i32(ctx), lse=lse, **scales)
    sv.kv_weigh(q, k, pages, i32(ctx), lse, w, k_scale=scales.get("k_scale"))
    rows = T * Hq // H
    assert ((w.double().view(B, maxp, H, page).sum((1, 3)) - rows).abs() <= rows * 2.0 ** -12).all()


@pytest.mark.parametrize("kind", ["e4m3", "pages"])
@pytest.mark.parametrize("Hq,D", [(2, 64), (8, 128), (40, 64), (64, 128)])
@pytest.mark.parametrize("large", [100.0, 700.0])
def test_weights_with_a_large_query_channel(kind, Hq, D, large):
    """One channel that is far above the others, which is usual: over E4M3 keys an element is off by 2^-21 of its row's largest, and a
    score by that times the sum of its key's elements; the sums of attention and the weights are held to it."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(Hq)
    B, T, H, page, ctx = 2, 3, 2, 16, [40, 1900]
    maxp = -(-(max(ctx) + T) // page)
    k, v, scales, *_ = cache(kind, B * maxp, page, H, D, g)
    if kind == "pages":  # so that scores of the usual size come out
        scales["k_scale"].fill_(2.0 ** -7)
    q = torch.randn((B, T, Hq, D), generator=g)
    q[..., 5] = large
    q = q.to(BF)
    k.view(torch.uint8)[..., 5] = 8 + torch.randint(0, 2, k.shape[:-1], generator=g).to(torch.uint8)  # 2^-6 and a step more
    kv = P.values(k, scales["k_scale"].cpu()) if kind == "pages" else k.contiguous().view(torch.uint8).view(R.F8).double() * scales["k_scale"].cpu().double()[:, None]
    pages, scale, tb = R.tables(B, maxp, B * maxp, g), D ** -0.5, [T] * B
    lse = torch.zeros((B, T, Hq), device="cuda")
    args = pages.cuda(), i32(ctx)
    sv.paged_attention(q.cuda(), R.to_cuda(k), R.to_cuda(v), *args, lse=lse, **scales)
    want, bound = P.lse(q, kv, pages, ctx, tb, None, scale, False)
    extra = torch.zeros(kv.shape[:1] + (H, page), dtype=torch.float64)
    for b, t, n, z, _ in P.scores(q, kv, pages, ctx, tb, None, scale, False):
        kk = kv[pages[b].long()[n // page], n % page].transpose(0, 1)
        top = q[b, t].double().abs().view(H, Hq // H, D).amax(-1)[..., None]
        off = 2.0 ** -21 * top * kk.abs().sum(-1)[:, None] * scale
        bound[b, t] += off.amax(-1).view(-1)
        w = torch.exp(z - want[b, t].view(H, -1, 1))
        extra[pages[b].long()[n // page], :, n % page] += (w * torch.expm1(off)).sum(1).T
    off = (lse.cpu().double() - want).abs()
    assert (off <= bound).all(), f"lse over the bound by {(off / bound).max():.3g} times"
    given, weight = want.float(), torch.zeros(extra.shape)
    w = weight.cuda()
    sv.kv_weigh(q.cuda(), R.to_cuda(k), *args, given.cuda(), w, k_scale=scales["k_scale"])
    want, _, bound = P.weigh(q, kv, pages, ctx, tb, None, scale, given, weight, torch.zeros(weight.shape, dtype=torch.int32), None, False)
    off = (w.cpu().double() - want).abs()
    assert (off <= bound + extra).all(), f"weights over the bound by {(off / (bound + extra)).nan_to_num().max():.3g} times"


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq", [2, 40])
def test_a_sum_that_is_nan_shows_where_its_row_attends(kind, Hq):
    """As after a wait that gave up: the row's weights are NaN, and slots that it does not attend to have none of it."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(2)
    B, T, H, D, page, ctx = 2, 3, 2, 64, 16, [30, 300]
    maxp = -(-(max(ctx) + T) // page)
    k, v, scales, *_ = cache(kind, B * maxp, page, H, D, g)
    k, v, pages, n = R.to_cuda(k), R.to_cuda(v), R.tables(B, maxp, B * maxp, g), i32(ctx)
    q, lse = torch.randn((B, T, Hq, D), generator=g).to(BF).cuda(), torch.zeros((B, T, Hq), device="cuda")
    sv.paged_attention(q, k, v, pages.cuda(), n, lse=lse, **scales)
    both = []
    for bad in (False, True):
        if bad:
            lse[1, 1, 0] = math.nan  # request 1, head 0: the context, tokens 0 and 1
        w = torch.zeros((B * maxp, H, page), device="cuda")
        sv.kv_weigh(q, k, pages.cuda(), n, lse, w, k_scale=scales.get("k_scale"))
        both.append(w.cpu())
    lost = torch.zeros(both[0].shape, dtype=torch.bool)
    for s in range(ctx[1] + 2):
        p, r = R.at(pages, 1, s, page)
        lost[p, 0, r] = True
    assert torch.equal(torch.isnan(both[1]), lost) and torch.equal(both[0][~lost], both[1][~lost])


@pytest.mark.parametrize("kind", KINDS)
def test_attention_and_weigh_captured_and_on_another_stream(kind):
    """Both as one graph that is replayed on other queries, and on a stream of their own, give what the calls give."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(9)
    B, T, Hq, H, D, page, ctx = 3, 4, 12, 2, 64, 16, [1500, 33, 700]
    maxp = -(-(max(ctx) + T) // page)
    k, v, scales, *_ = cache(kind, B * maxp, page, H, D, g)
    k, v, pages, n = R.to_cuda(k), R.to_cuda(v), R.tables(B, maxp, B * maxp, g).cuda(), i32(ctx)
    q = torch.zeros((B, T, Hq, D), dtype=BF, device="cuda")

    def step(w, p, stream=None):
        lse = torch.zeros((B, T, Hq), device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        out = sv.paged_attention(q, k, v, pages, n, lse=lse, stream=stream, **scales)
        sv.kv_weigh(q, k, pages, n, lse, w, p, k_scale=scales.get("k_scale"), stream=stream)
        return out, lse

    record = lambda: (torch.zeros((B * maxp, H, page), device="cuda"), torch.zeros((B * maxp, H, page), dtype=torch.int32, device="cuda"))  # noqa: E731
    side = torch.cuda.Stream()
    mine, twin, third = record(), record(), record()
    with torch.cuda.stream(side):
        step(*record())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = step(*mine)
    for seed in range(3):
        q.copy_(torch.randn(q.shape, generator=g) * (1 + seed))
        graph.replay()
        want = step(*twin)
        torch.cuda.synchronize()
        other = step(*third, stream=side)
        torch.cuda.synchronize()
        for x, y, z in zip((out, lse, *mine), (*want, *twin), (*other, *third)):
            assert torch.equal(x, y) and torch.equal(x, z)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("Hq", [8, 84])
def test_a_callers_workspace_of_just_the_size(kind, Hq):
    """With sums, over a table that cuts items: nothing behind the workspace's bytes is written, and less is refused."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(1)
    B, T, H, D, page, ctx = 2, 3, 2, 128, 16, [1900, 40]
    maxp = -(-(max(ctx) + T) // page)
    k, v, scales, *_ = cache(kind, B * maxp, page, H, D, g)
    k, v, pages, n = R.to_cuda(k), R.to_cuda(v), R.tables(B, maxp, B * maxp, g).cuda(), i32(ctx)
    q = torch.randn((B, T, Hq, D), generator=g).to(BF).cuda()
    size = sv.load().spec_paged_attention_workspace_bytes(B, T, Hq, H, D)
    raw = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    lse, mine = torch.zeros((B, T, Hq), device="cuda"), torch.zeros((B, T, Hq), device="cuda")
    want = sv.paged_attention(q, k, v, pages, n, lse=lse, **scales)
    got = sv.paged_attention(q, k, v, pages, n, lse=mine, workspace_tensor=raw[:size], **scales)
    assert torch.equal(got, want) and torch.equal(mine, lse) and (raw[size:] == 0xA5).all()
    with pytest.raises(sv.SpecVerifyError):
        sv.paged_attention(q, k, v, pages, n, lse=mine, workspace_tensor=raw[:size - 256], **scales)


# ------------------------------------------------------------------------------------------------
# selection and moves
# ------------------------------------------------------------------------------------------------
def record(B, H, page, slots, g, layers=None):
    maxp = -(-slots // page)
    num = B * maxp + 2
    shape = (() if layers is None else (layers,)) + (num, H, page)
    return torch.rand(shape, generator=g) ** 8, torch.randint(0, 2 * slots, shape, generator=g).to(torch.int32), R.tables(B, maxp, num, g)


def same_lists(a, b):
    (s1, t1, n1, m1), (s2, t2, n2, m2) = a, b
    assert torch.equal(n1, n2) and torch.equal(m1, m2)
    counts = torch.arange(s1.shape[-1], device="cuda") < n1[..., None]
    assert torch.equal(s1[counts], s2[counts]) and torch.equal(t1[counts], t2[counts])


@pytest.mark.parametrize("layers,B,H,slots", [(None, 1, 1, 40000), (4, 16, 8, 3000), (2, 300, 2, 100)])
@pytest.mark.parametrize("which", ["ctx", "budget", "seen"])
def test_select_replaces_lengths_in_place(layers, B, H, slots, which):
    """The new lengths go to an input that every list's blocks read: the lists are those of a call with a tensor of its own."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(2)
    w, p, pages = (x.cuda() for x in record(B, H, 16, slots, g, layers))
    ctx = torch.randint(slots // 2, slots + 1, (B,), generator=g)
    given = dict(ctx=ctx, budget=torch.randint(0, slots // 2, (B,), generator=g), seen=ctx + 7)
    given = {n: x.to(torch.int32).cuda() for n, x in given.items()}
    want = sv.kv_select(w, p, pages, given["ctx"], given["budget"], seen=given["seen"], first=2, recent=30)
    before = {n: x.clone() for n, x in given.items()}
    for _ in range(3):
        for n, x in given.items():
            x.copy_(before[n])
        out = tuple(torch.full_like(x, -1) for x in want[:3]) + (given[which],)
        got = sv.kv_select(w, p, pages, given["ctx"], given["budget"], seen=given["seen"], first=2, recent=30, out=out)
        assert got[3] is given[which]
        same_lists(got, want)
        for n, x in given.items():
            assert torch.equal(x, want[3] if n == which else before[n])


def test_a_loop_that_evicts_in_place_captured_and_replayed():
    """Selection, move and the next tokens' lengths as one graph over the same ctx_len."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(6)
    B, H, D, page, slots = 6, 4, 64, 16, 400
    w, p, pages = record(B, H, page, slots, g)
    k, v = (torch.randn((w.shape[0], page, H, D), generator=g).to(BF).cuda() for _ in range(2))
    dev, pages, budget = [k, v, w.cuda(), p.cuda()], pages.cuda(), i32([100, 1, 0, 399, 64, 200])
    start = [400, 300, 17, 400, 65, 399]

    def step(x, ctx, out):
        got = sv.kv_select(x[2], x[3], pages, ctx, budget, out=out)
        sv.kv_move(x[0], x[1], pages, got[3], *got[:3], weight=x[2], position=x[3])
        ctx += 3
        return got

    most = pages.shape[1] * page // 2
    lists = lambda: [torch.zeros((B, H, most), dtype=torch.int32, device="cuda") for _ in range(2)] + [torch.zeros((B, H), dtype=torch.int32, device="cuda")]  # noqa: E731
    ctx, mine = i32(start), lists()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        warm = i32(start)
        step([x.clone() for x in dev], warm, (*lists(), warm))
    torch.cuda.current_stream().wait_stream(side)
    twin = [x.clone() for x in dev]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(dev, ctx, (*mine, ctx))
    ctx.copy_(i32(start))
    other = i32(start)
    for _ in range(4):
        graph.replay()
        new = torch.zeros_like(other)
        step(twin, other, (*lists(), new))  # lengths of their own
        other = new + 3
        torch.cuda.synchronize()
        assert torch.equal(ctx, other)
        for x, y in zip(dev, twin):
            assert torch.equal(x, y)


@pytest.mark.parametrize("end", [203, 201])
@pytest.mark.parametrize("behind", [29, 33, 64, 150])
def test_move_with_many_left_out_behind_the_last_page(end, behind):
    """A short last page, whose rows behind the end go to other pages, and behind its own moves many that are left out for their
    targets: every entry keeps its value, whatever the pages' scales."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(end + behind)
    B, H, D, page, slots = 3, 2, 64, 8, 500
    w, pos, pages = record(B, H, page, slots, g)
    k, v, ks, vs = P.pool(w.shape[0], page, H, D, "slot", g)
    ks, vs = (2.0 ** torch.randint(-20, 20, x.shape, generator=g).float() for x in (ks, vs))
    last = end // 8 * 8
    targets = sorted(torch.randperm(last, generator=g)[:90].tolist()) + list(range(last, end))
    sources = list(range(end, end + 8)) + sorted((end + 8 + torch.randperm(slots - end - 8, generator=g)[:len(targets) + behind - 8]).tolist())
    pairs = list(zip(sources, targets))
    n = len(sources)
    src, dst = (torch.tensor(x, dtype=torch.int32).expand(B, H, n).contiguous().cuda() for x in (sources, targets + list(range(end, end + behind))))
    dev = [R.to_cuda(k), R.to_cuda(v), ks.cuda(), vs.cuda(), w.cuda(), pos.cuda()]
    sv.kv_move(dev[0], dev[1], pages.cuda(), i32([end] * B), src, dst, torch.full((B, H), n, dtype=torch.int32, device="cuda"),
               k_scale=dev[2], v_scale=dev[3], weight=dev[4], position=dev[5])
    torch.cuda.synchronize()
    at = lambda b, s: (int(pages[b, s // page]), s % page)  # noqa: E731
    for b in range(B):
        for h in range(H):
            P.moved(k, ks, pages[b], pairs, h, end, page)
            P.moved(v, vs, pages[b], pairs, h, end, page)
            for s, t in pairs:
                for x in (w, pos):
                    x[at(b, t)[0], h, at(b, t)[1]] = x[at(b, s)[0], h, at(b, s)[1]]
    for got, want in zip(dev, (k, v, ks, vs, w, pos)):
        got = got.cpu()
        got, want = (x.view(torch.uint8) if x.dtype == R.F8 else x for x in (got, want))
        assert torch.equal(got, want), int((got != want).sum())
