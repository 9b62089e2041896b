"""An E4M3 cache with a scale per page and head: paged_attention over it, kv_append and kv_keep that set it, against the
definitions in 64 bits.  Codes and scales are compared exactly where the arithmetic has few enough bits."""
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
# attention
# ------------------------------------------------------------------------------------------------
def build(B, T, Hq, H, D, page, ctx, layout="slot", seed=1, mask=None, tb=None, garbage=True, spread=3):
    g = torch.Generator().manual_seed(seed)
    max_pages = -(-(max(ctx) + T) // page) + 1
    num_pages = B * max_pages + 2
    k, v, ks, vs = P.pool(num_pages, page, H, D, layout, g, spread=spread)
    pages = R.tables(B, max_pages, num_pages, g)
    tb = [T] * B if tb is None else tb
    if garbage:  # NaN codes, and scales that do not count, everywhere that holds no token
        used = torch.zeros((num_pages, page), dtype=torch.bool)
        for b in range(B):
            for s in range(ctx[b] + tb[b]):
                used[R.at(pages, b, s, page)] = True
        for c in (k, v):
            c.view(torch.uint8)[~used] = 0x7F
        for s in (ks, vs):
            s[~used.any(1)] = math.nan
        for b in range(B):
            pages[b, -(-(ctx[b] + tb[b]) // page):] = 2 ** 30 + b
    q = (torch.randn((B, T, Hq, D), generator=g) * 1.5).to(BF)
    return dict(q=q, k=k, v=v, ks=ks, vs=vs, pages=pages, ctx=ctx, tb=tb, mask=mask, scale=D ** -0.5)


def call(d, lse=True, ragged=True, **kw):
    import speculative_decoding_rejection_verify_gb300 as sv
    sums = torch.full(d["q"].shape[:3], math.nan, device="cuda") if lse else None
    out = sv.paged_attention(d["q"].cuda(), R.to_cuda(d["k"]), R.to_cuda(d["v"]), d["pages"].cuda(), i32(d["ctx"]),
                             i32(d["tb"]) if ragged else None, mask=None if d["mask"] is None else d["mask"].cuda(),
                             scale=d["scale"], k_scale=d["ks"].cuda(), v_scale=d["vs"].cuda(), lse=sums, **kw)
    torch.cuda.synchronize()
    return (out, sums) if lse else out


def check(d, **kw):
    out, sums = call(d, **kw)
    k, v = (torch.nan_to_num(P.values(d[n], d[n + "s"])) for n in "kv")
    want, bound = R.attention(d["q"], k, v, d["pages"], d["ctx"], d["tb"], d["mask"], d["scale"])
    off = (out.cpu().double() - want).abs()
    assert (off <= bound).all(), f"over the bound by {(off - bound).max():.3g}"
    want, bound = P.lse(d["q"], k, d["pages"], d["ctx"], d["tb"], d["mask"], d["scale"], True)
    got = sums.cpu().double()
    assert torch.equal(torch.isinf(got), torch.isinf(want))
    off = torch.where(torch.isinf(want), 0.0, (got - torch.nan_to_num(want, neginf=0.0)).abs())
    assert (off <= bound).all(), f"lse over the bound by {(off - bound).max():.3g}"
    return out, sums


@pytest.mark.parametrize("T,Hq,H,D", [(1, 1, 1, 64), (1, 8, 8, 128), (1, 8, 2, 64), (5, 8, 2, 128), (6, 7, 1, 128),
                                      (3, 15, 5, 64), (17, 8, 1, 128), (9, 12, 1, 64), (17, 8, 2, 64), (64, 6, 2, 128),
                                      (1, 128, 1, 128), (33, 4, 4, 128), (64, 12, 2, 64)])
def test_head_layouts(T, Hq, H, D):
    check(build(2, T, Hq, H, D, 16, [37, 300]))


@pytest.mark.parametrize("ctx", [0, 1, 7, 15, 16, 63, 64, 126, 127, 128, 129, 255, 256, 383, 640])
def test_lengths_around_every_boundary(ctx):
    check(build(1, 3, 4, 2, 128, 16, [ctx], seed=ctx))
    check(build(1, 1, 2, 1, 64, 32, [ctx], "head", seed=ctx), ragged=False)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("layout", ["slot", "head"])
def test_page_sizes_and_orders(page, layout):
    check(build(3, 4, 8, 2, 128, page, [5, 130, 517], layout, seed=page))
    check(build(2, 2, 4, 2, 64, page, [1, 260], layout, seed=page))


def test_ragged_batch_with_empty_requests():
    ctx, tb = [0, 5, 900, 0, 64, 2000, 1, 130], [0, 3, 0, 5, 1, 5, 2, 4]
    out, sums = check(build(8, 5, 8, 2, 128, 16, ctx, tb=tb))
    for b, n in enumerate(tb):
        assert (out[b, n:] == 0).all() and (sums[b, n:] == -math.inf).all()


@pytest.mark.parametrize("width", [1, 40, 4000])
def test_the_page_tables_width_changes_nothing(width):
    """A wide table cuts items over the SMs and joins them."""
    d = build(3, 4, 8, 2, 128, 16, [5, 700, 1900])
    d["pages"] = torch.cat([d["pages"], torch.full((3, width), -7, dtype=torch.int32)], 1)
    check(d)


@pytest.mark.parametrize("Hq,H", [(4, 2), (32, 2), (48, 1), (64, 1)])
def test_trees_and_rows_that_attend_to_nothing(Hq, H):
    g = torch.Generator().manual_seed(Hq)
    B, T = 3, 2 if Hq == 64 else 9
    mask = torch.randint(0, 1 << T, (B, T), generator=g, dtype=torch.int64)
    mask[0, 0] = 0
    d = build(B, T, Hq, H, 128, 16, [0, 200, 33], mask=mask)
    out, sums = check(d)
    assert (out[0, 0] == 0).all() and (sums[0, 0] == -math.inf).all()


def test_scales_far_apart():
    """Pages at 2^-24 and 2^24 of one another's scale: a value's share goes by weight times scale, the sum by the weight."""
    d = build(2, 3, 8, 2, 64, 16, [190, 460])
    g = torch.Generator().manual_seed(5)
    pick = torch.randint(0, 3, d["vs"].shape, generator=g)
    d["vs"] = torch.where(torch.isnan(d["vs"]), d["vs"], torch.tensor([2.0 ** -24, 1.0, 2.0 ** 24])[pick])
    d["ks"] = torch.where(torch.isnan(d["ks"]), d["ks"], torch.full_like(d["ks"], 2.0 ** -9))
    # fp16 weights reach down to 2^-31 of the largest weight x scale, codes reach 448: below the bound's 2^-24 of the largest value
    check(d)


def test_scales_that_are_no_powers_of_two():
    d = build(2, 3, 8, 2, 128, 32, [190, 460])
    g = torch.Generator().manual_seed(6)
    for n in ("ks", "vs"):
        d[n] = d[n] * (torch.rand(d[n].shape, generator=g) + 0.5)
    check(d)


@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, 0.0, -1.0, 2.0 ** 25, 2.0 ** -25])
@pytest.mark.parametrize("Hq", [4, 48])
def test_a_scale_that_does_not_count(which, bad, Hq):
    """NaN for the rows that attend to a slot of the page, nothing for the others."""
    T = 4
    mask = torch.tensor([[1, 2, 4, 9]], dtype=torch.int64)  # token 3 attends to itself and token 0
    d = build(1, T, Hq, 2, 64, 8, [13], mask=mask, garbage=False)  # slots 13, 14, 15 | 16: token 3's slot begins page 2
    d[which][d["pages"][0, 2], 1] = bad
    out, sums = call(d)
    G = Hq // 2
    assert torch.isnan(out[0, 3, G:]).all() and not torch.isnan(out[0, 3, :G]).any() and not torch.isnan(out[0, :3]).any()
    assert torch.isnan(sums[0, 3, G:]).all()
    clean = build(1, T, Hq, 2, 64, 8, [13], mask=mask, garbage=False)
    ref, ref_sums = call(clean)
    assert torch.equal(out[0, :3], ref[0, :3]) and torch.equal(sums[0, :3], ref_sums[0, :3])


def test_pages_outside_the_pool_read_as_zeros():
    d = build(1, 2, 4, 2, 64, 16, [60], garbage=False)
    d["pages"][0, 1], d["pages"][0, 2] = -3, 2 ** 30
    out, sums = call(d)
    k, v = P.values(d["k"], d["ks"]), P.values(d["v"], d["vs"])
    zero = torch.zeros((1,) + k.shape[1:], dtype=torch.float64)
    k, v = torch.cat([k, zero]), torch.cat([v, zero])
    pages = torch.where((d["pages"] < 0) | (d["pages"] > k.shape[0]), k.shape[0] - 1, d["pages"])
    want, bound = R.attention(d["q"], k, v, pages, d["ctx"], d["tb"], None, d["scale"])
    assert ((out.cpu().double() - want).abs() <= bound).all()


@pytest.mark.parametrize("dtype", [BF, R.F8])
@pytest.mark.parametrize("Hq", [4, 40])
def test_lse_of_the_other_caches(dtype, Hq):
    """bf16: the sum is that of weights rounded to bf16, each within 2^-8, so the logarithm is within 2^-8 (1 + 2^-8)."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(3)
    B, T, H, D, page, ctx = 2, 3, 2, 64, 16, [40, 700]
    k, v = R.pool(B * 45, page, H, D, dtype, "slot", g)
    pages = R.tables(B, 45, B * 45, g)
    q = torch.randn((B, T, Hq, D), generator=g).to(BF)
    ks = torch.rand(H, generator=g) + 0.5 if dtype == R.F8 else None
    sums = torch.zeros((B, T, Hq), device="cuda")
    args = (q.cuda(), R.to_cuda(k), R.to_cuda(v), pages.cuda(), i32(ctx))
    out = sv.paged_attention(*args, k_scale=R.to_cuda(ks), lse=sums)
    assert torch.equal(out, sv.paged_attention(*args, k_scale=R.to_cuda(ks)))
    values = k.contiguous().view(torch.uint8).view(R.F8).double() * ks.double()[:, None] if dtype == R.F8 else k.double()
    want, bound = P.lse(q, values, pages, ctx, [T] * B, None, D ** -0.5, dtype == R.F8)
    bound = bound + (2.0 ** -8 * (1 + 2.0 ** -8) if dtype == BF else 0.0)
    assert ((sums.cpu().double() - want).abs() <= bound).all()


# ------------------------------------------------------------------------------------------------
# append
# ------------------------------------------------------------------------------------------------
def angles(n, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2).double() / rot)
    a = torch.arange(n).double()[:, None] * f
    return a.cos().float(), a.sin().float()


def turned(x, cos, sin, interleaved):
    """The rotation as the cache's keys take it: fp32 products and their fp32 sum, each rounded (so exactly comparable)."""
    r = 2 * len(cos)
    x = x.float()
    y = x.clone()
    i = torch.arange(r // 2)
    a, c = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    y[..., a] = x[..., a] * cos - x[..., c] * sin
    y[..., c] = x[..., c] * cos + x[..., a] * sin
    return y


class Cache:
    """A cache with page scales on the GPU, and what it has to hold."""

    def __init__(self, B, H, D, page, slots, layout="slot", seed=1, layers=None):
        self.g = torch.Generator().manual_seed(seed)
        self.page, self.H, self.D, self.B = page, H, D, B
        max_pages = -(-slots // page)
        self.k, self.v, self.ks, self.vs = P.pool(B * max_pages + 2, page, H, D, layout, self.g, layers)
        self.pages = R.tables(B, max_pages, B * max_pages + 2, self.g)
        self.dev = [R.to_cuda(self.k), R.to_cuda(self.v), self.ks.cuda(), self.vs.cuda()]
        # the references index [pages, page, heads, D] and may change in place
        self.k, self.v = self.k.contiguous(), self.v.contiguous()

    def same(self):
        torch.cuda.synchronize()
        for got, want in zip(self.dev, (self.k, self.v, self.ks, self.vs)):
            got = got.cpu()
            if got.dtype == R.F8:
                got, want = got.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8)
                nan = ((got & 0x7F) == 0x7F) & ((want & 0x7F) == 0x7F)
                got, want = torch.where(nan, 0, got), torch.where(nan, 0, want)
            assert torch.equal(got, want), (got != want).sum()

    def append(self, q, k, v, ctx, rot=0, interleaved=False, tb=None, positions=None, **kw):
        import speculative_decoding_rejection_verify_gb300 as sv
        B, T = k.shape[:2]
        cos, sin = angles(max(ctx) + T + 5, rot) if rot else (None, None)
        up = lambda x: None if x is None else x.cuda()  # noqa: E731
        out = sv.kv_append(up(q), k.cuda(), v.cuda(), self.dev[0], self.dev[1], self.pages.cuda(), i32(ctx), up(cos), up(sin),
                           None if tb is None else i32(tb), positions=up(positions), interleaved=interleaved,
                           k_scale=self.dev[2], v_scale=self.dev[3], **kw)
        for b in range(B):
            n = T if tb is None else min(max(tb[b], 0), T)
            at = [ctx[b] + t if positions is None else int(positions[b, t]) for t in range(n)]
            kk = torch.stack([turned(k[b, t], cos[at[t]], sin[at[t]], interleaved) if rot else k[b, t].float() for t in range(n)]) if n else None
            for p in range(ctx[b] // self.page, -(-(ctx[b] + n) // self.page) if n else 0):
                here = [t for t in range(n) if (ctx[b] + t) // self.page == p]
                if not here:
                    continue
                stays = list(range(ctx[b] - p * self.page)) if p * self.page < ctx[b] else None
                for h in range(self.H):
                    for cache, scale, x in ((self.k, self.ks, kk), (self.v, self.vs, v[b].float())):
                        P.put(cache, scale, int(self.pages[b, p]), h, [(ctx[b] + t) % self.page for t in here], x[here, h].double(), stays)
        return out


def tokens(B, T, Hq, H, D, g, sd=1.0):
    n = Hq + 2 * H
    x = torch.randn((B, T, n, D), generator=g) * sd * torch.exp(torch.randn((B, T, n, 1), generator=g))
    x = x.to(BF)
    return x[:, :, :Hq], x[:, :, Hq:Hq + H], x[:, :, Hq + H:]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 32), (64, 16), (128, 0), (128, 48)])
def test_append_rotations(D, rot, interleaved):
    c = Cache(3, 2, D, 16, 760)
    q, k, v = tokens(3, 4, 6, 2, D, c.g)
    out = c.append(q, k, v, [0, 13, 700], rot, interleaved)
    c.same()
    cos, sin = angles(760, max(rot, 2))
    for b, n in enumerate([0, 13, 700]):
        for t in range(4):
            want, e = R.rotate(q[b, t].double(), cos[n + t].double().tolist() if rot else [], sin[n + t].double().tolist() if rot else [], interleaved)
            assert ((out[b, t].cpu().double() - want).abs() <= R.U_BF16 * want.abs() + e).all()


@pytest.mark.parametrize("page", [8, 16, 32, 64, 256, 4096])
@pytest.mark.parametrize("layout", ["slot", "head"])
def test_append_pages(page, layout):
    c = Cache(2, 3, 64, page, 900, layout, seed=page)
    _, k, v = tokens(2, 150, 0, 3, 64, c.g)
    c.append(None, k, v, [5, 700], 64, tb=[150, 77])
    c.same()


def test_append_step_by_step():
    """A page's scale grows over the steps, and what it holds follows."""
    c = Cache(4, 2, 64, 16, 120)
    ctx = [0, 3, 15, 16]
    for step in range(12):
        _, k, v = tokens(4, 5, 0, 2, 64, c.g, 2.0 ** (step % 5))
        tb = [5, step % 6, 1, 0]
        c.append(None, k, v, ctx, 32, tb=tb)
        c.same()
        ctx = [n + t for n, t in zip(ctx, tb)]


def test_append_many_tokens():
    """More tokens of a page than a thread holds, and more pages than a block."""
    c = Cache(1, 1, 128, 512, 3000)
    _, k, v = tokens(1, 2500, 0, 1, 128, c.g)
    c.append(None, k, v, [77], 128, interleaved=True)
    c.same()


def test_append_odd_values():
    """Zeros, infinities, NaN, the largest and smallest magnitudes, and amounts on either side of a power's border."""
    c = Cache(1, 6, 64, 8, 64)
    _, k, v = tokens(1, 8, 0, 6, 64, c.g)
    k, v = k.clone(), v.clone()
    k[0, :, 0] = 0.0
    k[0, 3, 1, 5], k[0, 4, 1, 6], k[0, 5, 1, 7] = math.inf, -math.inf, math.nan
    k[0, :, 2] *= 2.0 ** 60
    k[0, :, 3] *= 2.0 ** -60
    v[0, :, 4] = v[0, :, 4].clamp(-448, 448)
    v[0, 2, 4, 9] = 448.0
    v[0, :, 5] = v[0, :, 5].clamp(-448, 448)
    v[0, 2, 5, 9] = 450.0
    v[0, :, 0] = math.nan
    v[0, :, 1] = -math.inf
    c.append(None, k, v, [24])
    c.same()
    assert float(c.vs[c.pages[0, 3], 4]) == 1.0 and float(c.vs[c.pages[0, 3], 5]) == 2.0
    assert float(c.ks[c.pages[0, 3], 2]) == 2.0 ** 24 and float(c.ks[c.pages[0, 3], 0]) == 2.0 ** -24


@pytest.mark.parametrize("old", [math.nan, 0.0, -2.0, math.inf, 2.0 ** 30, 0.37])
def test_append_behind_a_scale_that_does_not_count_or_is_no_power(old):
    """One that does not count is replaced and the codes before are left alone; 0.37 counts: codes are round(x / 0.37)."""
    c = Cache(1, 1, 64, 16, 32)
    for s, d in ((c.ks, c.dev[2]), (c.vs, c.dev[3])):
        s[c.pages[0, 0], 0] = old
        d[c.pages[0, 0].item(), 0] = old
    _, k, v = tokens(1, 3, 0, 1, 64, c.g)
    c.append(None, k, v, [5])
    if old == 0.37:  # the reference's quotient has 53 bits, the kernel's is correctly rounded to 24: at most a code apart, on a tie
        torch.cuda.synchronize()
        got, want = c.dev[0].cpu().view(torch.uint8).int(), c.k.view(torch.uint8).int()
        assert (got - want).abs().max() <= 1 and ((got != want).sum() <= 1)
        assert torch.equal(c.dev[2].cpu(), c.ks)
    else:
        c.same()


def test_append_trees_and_flags():
    import speculative_decoding_rejection_verify_gb300 as sv
    c = Cache(3, 2, 64, 16, 96)
    q, k, v = tokens(3, 7, 4, 2, 64, c.g)
    positions = torch.tensor([[5 + d for d in (0, 1, 2, 1, 2, 1, 2)]] * 3, dtype=torch.int32)
    flags = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = c.append(q, k, v, [5, 60, 90], 64, positions=positions, tb=[7, 2, 0], flags=flags)
    c.same()
    assert (flags == 0).all() and (out[2] == 0).all() and (out[1, 2:] == 0).all()
    # beyond the table, a bad page, a bad count: flagged, and nothing outside is written
    before = [x.clone() for x in c.dev]
    pages = c.pages.clone()
    pages[1] = -1
    sv.kv_append(None, k.cuda(), v.cuda(), c.dev[0], c.dev[1], pages.cuda(), i32([96, 0, 10]), None, None, i32([7, 7, -4]),
                 k_scale=c.dev[2], v_scale=c.dev[3], flags=flags)
    torch.cuda.synchronize()
    assert flags.tolist() == [sv.FLAG_BAD_SLOT, sv.FLAG_BAD_SLOT, sv.FLAG_BAD_K]
    for x, y in zip(c.dev, before):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_append_across_the_tables_end():
    """The tokens that the table still holds go in; a page's scale follows those alone that are in it."""
    c = Cache(1, 1, 64, 8, 24)
    _, k, v = tokens(1, 6, 0, 1, 64, c.g)
    import speculative_decoding_rejection_verify_gb300 as sv
    sv.kv_append(None, k.cuda(), v.cuda(), c.dev[0], c.dev[1], c.pages.cuda(), i32([21]), k_scale=c.dev[2], v_scale=c.dev[3])
    for cache, scale, x in ((c.k, c.ks, k), (c.v, c.vs, v)):
        P.put(cache, scale, int(c.pages[0, 2]), 0, [5, 6, 7], x[0, :3, 0].double(), range(5))
    c.same()


# ------------------------------------------------------------------------------------------------
# keep
# ------------------------------------------------------------------------------------------------
def run_keep(c, ctx, path, n, layers, record=False):
    import speculative_decoding_rejection_verify_gb300 as sv
    shape = c.dev[0].shape[:-3] + (c.H, c.page)
    w = torch.rand(shape, generator=c.g)
    pos = torch.randint(0, 9999, shape, generator=c.g).to(torch.int32)
    extra = dict(weight=w.cuda(), position=pos.cuda()) if record else {}
    sv.kv_keep(c.dev[0], c.dev[1], c.pages.cuda(), i32(ctx), path.cuda(), i32(n), k_scale=c.dev[2], v_scale=c.dev[3], **extra)
    side = lambda x, layer: x if layers is None else x[layer]  # noqa: E731
    for layer in range(layers or 1):
        for b, m in enumerate(n):
            m = min(max(m, 0), path.shape[1])
            pairs = [(ctx[b] + int(p), ctx[b] + i) for i, p in enumerate(path[b, :m]) if int(p) != i]
            for h in range(c.H):
                if pairs:
                    for cache, scale in ((c.k, c.ks), (c.v, c.vs)):
                        P.moved(side(cache, layer), side(scale, layer), c.pages[b], pairs, h, ctx[b] + m, c.page)
                for s, t in pairs:
                    for x in (w, pos):
                        y = side(x, layer)
                        y[c.pages[b, t // c.page], h, t % c.page] = y[c.pages[b, s // c.page], h, s % c.page]
    c.same()
    if record:
        assert torch.equal(extra["weight"].cpu(), w) and torch.equal(extra["position"].cpu(), pos)


def paths(B, T, most, g):
    out = torch.zeros((B, most), dtype=torch.int32)
    for b in range(B):
        out[b] = torch.sort(torch.randperm(T, generator=g)[:most]).values.to(torch.int32)
    return out


@pytest.mark.parametrize("layout", ["slot", "head"])
@pytest.mark.parametrize("page,D", [(8, 64), (16, 128), (64, 128), (512, 64)])
@pytest.mark.parametrize("layers", [None, 3])
def test_keep(page, D, layout, layers):
    c = Cache(5, 2, D, page, 400, layout, seed=page, layers=layers)
    path = paths(5, 33, 12, c.g)
    path[0] = torch.arange(12)  # nothing moves
    run_keep(c, [0, 7, 130, 254, 303], path, [12, 12, 5, 0, 9], layers, record=layers is not None)


def test_keep_of_64_entries_with_scales_far_apart():
    c = Cache(2, 3, 64, 8, 300)
    for s, d in ((c.ks, c.dev[2]), (c.vs, c.dev[3])):
        s.copy_(2.0 ** torch.randint(-20, 20, s.shape, generator=c.g).float())
        d.copy_(s)
    run_keep(c, [3, 150], paths(2, 100, 64, c.g), [64, 61], None)


def test_keep_leaves_out_what_lies_outside():
    import speculative_decoding_rejection_verify_gb300 as sv
    c = Cache(2, 1, 64, 8, 40)
    pages = c.pages.clone()
    pages[1, 1:] = -1
    path = torch.tensor([[1, 2, 39, 2 ** 30], [1, 30, 31, 32]], dtype=torch.int32)
    sv.kv_keep(c.dev[0], c.dev[1], pages.cuda(), i32([20, 2]), path.cuda(), i32([4, 4]), k_scale=c.dev[2], v_scale=c.dev[3])
    for cache, scale in ((c.k, c.ks), (c.v, c.vs)):
        P.moved(cache, scale, c.pages[0], [(21, 20), (22, 21)], 0, 24, 8)
        P.moved(cache, scale, c.pages[1], [(3, 2)], 0, 6, 8)
    c.same()


# ------------------------------------------------------------------------------------------------
# streams, graphs, threads
# ------------------------------------------------------------------------------------------------
def test_a_decode_step_captured_and_replayed():
    """append, attend, keep as one graph, replayed on new inputs, gives what the calls give."""
    import speculative_decoding_rejection_verify_gb300 as sv
    B, T, Hq, H, D, page = 3, 5, 8, 2, 64, 16
    c = Cache(B, H, D, page, 200)
    ctx, pages = i32([0, 30, 150]), c.pages.cuda()
    qkv = torch.zeros((B, T, Hq + 2 * H, D), dtype=BF, device="cuda")
    path, n = i32([[0, 3, 4], [1, 2, 3], [0, 1, 2]]), i32([3, 2, 3])
    lse = torch.zeros((B, T, Hq), device="cuda")

    def step(dev, lse):
        q = sv.kv_append(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:], dev[0], dev[1], pages, ctx, k_scale=dev[2], v_scale=dev[3])
        o = sv.paged_attention(q, dev[0], dev[1], pages, ctx, k_scale=dev[2], v_scale=dev[3], lse=lse)
        sv.kv_keep(dev[0], dev[1], pages, ctx, path, n, k_scale=dev[2], v_scale=dev[3])
        return o

    twin, lse2 = [x.clone() for x in c.dev], torch.zeros_like(lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step([x.clone() for x in c.dev], lse)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(c.dev, lse)
    for seed in range(3):
        torch.manual_seed(seed)
        qkv.copy_((torch.randn(qkv.shape) * 2.0 ** seed).to(BF))
        graph.replay()
        want = step(twin, lse2)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, lse2)
        for x, y in zip(c.dev, twin):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_on_another_stream():
    d = build(2, 3, 8, 2, 128, 16, [100, 1500])
    want, sums = call(d)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got, again = call(d, stream=stream)
    assert torch.equal(got, want) and torch.equal(sums, again)


def test_waits_that_give_up_leave_nan():
    """The waits' limit is set to one try: rows and their sums come out as NaN where a wait ran out, and later calls are whole."""
    import speculative_decoding_rejection_verify_gb300 as sv
    d = build(3, 4, 8, 2, 128, 16, [700, 1900, 300])
    want, sums = call(d)
    sv.set_test_hooks(2)
    try:
        out, lse = call(d)
    finally:
        sv.set_test_hooks(0)
    lost = torch.isnan(out).any(-1)
    assert lost.any()
    again, sums2 = call(d)
    assert torch.equal(again, want) and torch.equal(sums2, sums)


# ------------------------------------------------------------------------------------------------
# strides
# ------------------------------------------------------------------------------------------------
def far(x, stride):
    """x [pages, ...] with its pages `stride` bytes apart, so that offsets pass 32 bits."""
    n = x.shape[0]
    raw = torch.zeros(stride * (n - 1) + x[0].numel(), dtype=torch.uint8, device="cuda")
    y = raw.as_strided(x.shape, (stride,) + tuple(x.contiguous().stride()[1:])).view(R.F8)
    y.view(torch.uint8).copy_(x.view(torch.uint8))
    return y


def test_offsets_beyond_32_bits():
    """Append, attention, weigh, keep and move over pages 600 MB apart give what they give over adjacent ones."""
    import speculative_decoding_rejection_verify_gb300 as sv
    B, T, Hq, H, D, page = 1, 5, 8, 2, 64, 16
    c = Cache(B, H, D, page, 96)
    ctx, pages = i32([70]), c.pages.cuda()
    qkv = torch.randn((B, T, Hq + 2 * H, D), generator=c.g).to(BF).cuda()
    stride = 600 << 20
    results = []
    for pool in (c.dev[:2], [far(x, stride) for x in c.dev[:2]]):
        k, v, ks, vs = *pool, c.dev[2].clone(), c.dev[3].clone()
        if pool is c.dev[:2]:
            k, v = k.clone(), v.clone()
        q = sv.kv_append(qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:], k, v, pages, ctx, k_scale=ks, v_scale=vs)
        lse = torch.zeros((B, T, Hq), device="cuda")
        o = sv.paged_attention(q, k, v, pages, ctx, k_scale=ks, v_scale=vs, lse=lse)
        w, p = torch.zeros((k.shape[0], H, page), device="cuda"), torch.zeros((k.shape[0], H, page), dtype=torch.int32, device="cuda")
        sv.kv_weigh(q, k, pages, ctx, lse, w, p, k_scale=ks)
        sv.kv_keep(k, v, pages, ctx, i32([[0, 3, 4]]), i32([3]), k_scale=ks, v_scale=vs, weight=w, position=p)
        src, dst, n, m = sv.kv_select(w, p, pages, ctx + 3, i32([40]), recent=8)
        sv.kv_move(k, v, pages, m, src, dst, n, k_scale=ks, v_scale=vs, weight=w, position=p)
        torch.cuda.synchronize()
        results.append([o, lse, k.contiguous().view(torch.uint8), v.contiguous().view(torch.uint8), ks, vs, w, p, n, m])
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert int(results[0][8].sum()) > 0
