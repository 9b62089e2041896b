"""spec_paged_attention against the formula in float64: head layouts, lengths around every boundary, page
sizes and orders, trees, empty rows, garbage in every slot that is not attended to, streams, large pools.
The elementwise bound is derived in _decode.attention."""
import pytest
import torch

import _decode as R

pytestmark = pytest.mark.gpu


def build(B, T, Hq, H, D, page, ctx, dtype, layout, seed=1, mask=None, tb=None, garbage=True):
    g = torch.Generator().manual_seed(seed)
    need = max(ctx) + T
    max_pages = -(-need // page) + 1
    num_pages = B * max_pages + 2
    k, v = R.pool(num_pages, page, H, D, dtype, layout, g)
    pages = R.tables(B, max_pages, num_pages, g)
    tb = [T] * B if tb is None else tb
    if garbage:  # NaN everywhere that holds no token; page entries that hold none point outside the pool
        used = torch.zeros((num_pages, page), dtype=torch.bool)
        for b in range(B):
            for s in range(ctx[b] + tb[b]):
                used[R.at(pages, b, s, page)] = True
        for c in (k, v):
            raw = c.view(torch.uint8) if dtype == R.F8 else c
            raw[~used] = 0x7F if dtype == R.F8 else float("nan")
        for b in range(B):
            pages[b, -(-(ctx[b] + tb[b]) // page):] = 2 ** 30 + b
    q = (torch.randn((B, T, Hq, D), generator=g) * 2).to(torch.bfloat16)
    ks = vs = None
    if dtype == R.F8:
        ks, vs = torch.rand(H, generator=g) + 0.5, torch.rand(H, generator=g) + 0.5
    return dict(q=q, k=k, v=v, pages=pages, ctx=ctx, tb=tb, mask=mask, ks=ks, vs=vs, scale=D ** -0.5)


def call(d, ragged=True, **kw):
    import speculative_decoding_rejection_verify_gb300 as sv
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = sv.paged_attention(R.to_cuda(d["q"]), R.to_cuda(d["k"]), R.to_cuda(d["v"]), d["pages"].cuda(),
                             i32(d["ctx"]), i32(d["tb"]) if ragged else None,
                             mask=None if d["mask"] is None else d["mask"].cuda(), scale=d["scale"],
                             k_scale=R.to_cuda(d["ks"]), v_scale=R.to_cuda(d["vs"]), **kw)
    torch.cuda.synchronize()
    return out


def check(d, out=None, **kw):
    out = call(d, **kw) if out is None else out
    want, bound = R.attention(d["q"], d["k"], d["v"], d["pages"], d["ctx"], d["tb"], d["mask"], d["scale"], d["ks"],
                              d["vs"])
    got = out.cpu().double()
    assert torch.isfinite(got).all()
    off = (got - want).abs()
    worst = (off - bound).max()
    assert (off <= bound).all(), f"over the bound by {worst:.3g}, off by {off.max():.3g}"


BF = torch.bfloat16


@pytest.mark.parametrize("T,Hq,H,D", [(1, 1, 1, 64), (1, 8, 8, 128), (1, 8, 2, 64), (5, 8, 2, 128), (6, 7, 1, 128),
                                      (3, 15, 5, 64), (17, 8, 1, 128), (17, 16, 1, 64), (9, 12, 1, 64), (64, 6, 2, 128),
                                      (2, 64, 1, 64), (1, 128, 1, 128), (33, 4, 4, 128)])
@pytest.mark.parametrize("dtype", [BF, R.F8])
def test_head_layouts(T, Hq, H, D, dtype):
    check(build(2, T, Hq, H, D, 16, [37, 300], dtype, "slot"))


@pytest.mark.parametrize("ctx", [0, 1, 7, 15, 16, 63, 64, 111, 126, 127, 128, 129, 254, 255, 256, 383, 511, 640])
@pytest.mark.parametrize("dtype", [BF, R.F8])
def test_lengths_around_every_boundary(ctx, dtype):
    check(build(1, 3, 4, 2, 128, 16, [ctx], dtype, "slot", seed=ctx))
    check(build(1, 1, 2, 1, 64, 32, [ctx], dtype, "head", seed=ctx), ragged=False)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("layout", ["slot", "head"])
@pytest.mark.parametrize("dtype", [BF, R.F8])
def test_page_sizes_and_orders(page, layout, dtype):
    check(build(3, 4, 8, 2, 128, page, [5, 130, 517], dtype, layout, seed=page))
    check(build(2, 2, 4, 2, 64, page, [1, 260], dtype, layout, seed=page))


@pytest.mark.parametrize("dtype", [BF, R.F8])
def test_ragged_batch_with_empty_requests(dtype):
    ctx, tb = [0, 5, 900, 0, 64, 2000, 1, 130], [0, 3, 0, 5, 1, 5, 2, 4]
    d = build(8, 5, 8, 2, 128, 16, ctx, dtype, "slot", tb=tb)
    out = call(d)
    check(d, out)
    for b, n in enumerate(tb):
        assert (out[b, n:] == 0).all()


@pytest.mark.parametrize("dtype", [BF, R.F8])
def test_row_groups_without_tokens(dtype):
    """64 tokens of a wide group are several items; a request's few tokens leave the later ones without a row."""
    tb = [5, 64, 0, 33]
    d = build(4, 64, 12, 2, 64, 16, [130, 7, 50, 0], dtype, "slot", tb=tb)
    out = call(d)
    check(d, out)
    for b, n in enumerate(tb):
        assert (out[b, n:] == 0).all()


def test_queries_shared_by_the_batch():
    d = build(3, 2, 4, 2, 64, 16, [100, 7, 260], BF, "slot")
    d["q"] = d["q"][:1].expand(3, -1, -1, -1)
    import speculative_decoding_rejection_verify_gb300 as sv
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    q = d["q"][:1].cuda().expand(3, -1, -1, -1)
    out = sv.paged_attention(q, R.to_cuda(d["k"]), R.to_cuda(d["v"]), d["pages"].cuda(), i32(d["ctx"]))
    assert out.shape == q.shape
    check(d, out)


@pytest.mark.parametrize("dtype", [BF, R.F8])
@pytest.mark.parametrize("width", [1, 40, 4000])
def test_the_page_tables_width_changes_nothing(dtype, width):
    """A table that could hold many more pages takes the way over cut items; the result is the same."""
    d = build(3, 5, 8, 2, 128, 16, [300, 0, 77], dtype, "slot")
    d["pages"] = torch.cat([d["pages"], torch.full((3, width), 2 ** 30, dtype=torch.int32)], 1)
    check(d)


def test_values_that_are_not_finite_in_the_context():
    """A NaN in the context's values reaches every row of its heads and no other head or element."""
    d = build(1, 3, 4, 2, 64, 16, [200], BF, "slot", seed=8)
    want, bound = R.attention(d["q"], d["k"], d["v"], d["pages"], d["ctx"], d["tb"], None, d["scale"])
    p, r = R.at(d["pages"], 0, 60, 16)
    d["v"][p, r, 1, 5] = float("nan")
    got = call(d).cpu().double()
    hit = torch.zeros(got.shape, dtype=torch.bool)
    hit[0, :, 2:, 5] = True
    assert torch.isnan(got[hit]).all() and ((got - want).abs() <= bound)[~hit].all()


def test_many_requests_of_mixed_length():
    g = torch.Generator().manual_seed(9)
    ctx = torch.randint(0, 700, (90,), generator=g).tolist()
    check(build(90, 2, 4, 2, 64, 16, ctx, BF, "slot"))


@pytest.mark.parametrize("dtype", [BF, R.F8])
def test_long_cache_is_split_and_joined(dtype):
    check(build(1, 2, 4, 1, 128, 64, [40001], dtype, "head"))
    check(build(2, 1, 2, 2, 64, 16, [20000, 3], dtype, "slot"))


def tree(T, chains):
    import perf.operators as ops
    return ops._tree(T, chains)[1]


@pytest.mark.parametrize("T,chains,ctx", [(9, 2, [0, 120]), (17, 4, [126, 111]), (61, 4, [100, 65]), (64, 3, [64, 0])])
@pytest.mark.parametrize("dtype", [BF, R.F8])
def test_trees(T, chains, ctx, dtype):
    bits = tree(1 + (T - 1) // chains * chains, chains)
    bits += [-1] * (T - len(bits))  # the others attend to every new token
    check(build(2, T, 4, 2, 128, 16, ctx, dtype, "slot", mask=torch.tensor([bits, bits])))


def test_rows_that_attend_to_nothing_are_zero():
    mask = torch.tensor([[0, 1, 0, 1 << 3], [0, 0, 0, 0], [0, 2, 0, 0], [-1, -1, 0, 1]])
    d = build(4, 4, 4, 2, 128, 16, [0, 0, 20, 0], BF, "slot", mask=mask, tb=[4, 4, 4, 2])
    out = call(d)
    check(d, out)
    assert (out[0, 0] == 0).all() and (out[0, 2] == 0).all() and (out[1] == 0).all()


@pytest.mark.parametrize("dtype", [BF, R.F8])
@pytest.mark.parametrize("ctx", [0, 50, 125, 300])
def test_masked_tokens_hold_garbage(dtype, ctx):
    """NaN and infinities in a new token's K and V reach the rows that attend to it and no others."""
    T, bad = 6, 3
    for value in (float("nan"), float("inf")):
        if dtype == R.F8 and value == float("inf"):
            continue  # E4M3 has no infinity
        d = build(1, T, 4, 2, 128, 16, [ctx], dtype, "slot", seed=3)
        p, r = R.at(d["pages"], 0, ctx + bad, 16)
        clean = [c.clone() for c in (d["k"], d["v"])]
        for c in (d["k"], d["v"]):
            if dtype == R.F8:
                c.view(torch.uint8)[p, r] = 0x7F
            else:
                c[p, r] = value
        got = call(d)
        d["k"], d["v"] = clean
        want, bound = R.attention(d["q"], d["k"], d["v"], d["pages"], d["ctx"], d["tb"], None, d["scale"], d["ks"], d["vs"])
        assert ((got.cpu().double() - want).abs() <= bound)[:, :bad].all()
        if value != value:
            assert torch.isnan(got[:, bad:]).all()
    # V alone, one element: what attends to it gets that element, the others nothing of it
    d = build(1, T, 4, 2, 128, 16, [ctx], dtype, "slot", seed=4)
    p, r = R.at(d["pages"], 0, ctx + bad, 16)
    want, bound = R.attention(d["q"], d["k"], d["v"], d["pages"], d["ctx"], d["tb"], None, d["scale"], d["ks"], d["vs"])
    if dtype == R.F8:
        d["v"].view(torch.uint8)[p, r, 1, 77] = 0x7F
    else:
        d["v"][p, r, 1, 77] = float("-inf")
    got = call(d).cpu().double()
    hit = torch.zeros(got.shape, dtype=torch.bool)
    hit[0, bad:, 2:, 77] = True
    assert ((got - want).abs() <= bound)[~hit].all()
    assert (torch.isnan(got[hit]) if dtype == R.F8 else got[hit] == -float("inf")).all()


def test_large_scores_and_a_growing_maximum():
    """Scores that climb along the cache move the running maximum in every tile; huge ones do not overflow."""
    d = build(1, 2, 4, 2, 128, 16, [1000], BF, "slot", seed=5, garbage=False)
    ramp = torch.linspace(0.1, 12.0, 1002)
    for s in range(1002):
        p, r = R.at(d["pages"], 0, s, 16)
        d["k"][p, r] = (d["k"][p, r].float() * ramp[s]).to(BF)
    check(d)
    for s in range(1002):
        p, r = R.at(d["pages"], 0, s, 16)
        d["k"][p, r] = -(d["k"][p, r].float().abs() * 300 * d["q"][0, 0, 0].float().sign() * (0.5 + s / 1002)).to(BF)
    check(d)


def test_a_nan_query_spoils_its_own_row_only():
    d = build(1, 3, 2, 1, 64, 16, [200], BF, "slot", seed=6)
    d["q"][0, 1, 0] = float("nan")
    got = call(d).cpu()
    assert torch.isnan(got[0, 1, 0]).all()
    d["q"][0, 1, 0] = 0
    want, bound = R.attention(d["q"], d["k"], d["v"], d["pages"], d["ctx"], d["tb"], None, d["scale"])
    off = (got.double() - want).abs() <= bound
    assert off[0, 0].all() and off[0, 2].all() and off[0, 1, 1].all()


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scales(scale):
    d = build(2, 3, 4, 2, 64, 16, [100, 260], BF, "slot")
    d["scale"] = scale
    check(d)


def test_strided_queries_and_outputs():
    d = build(2, 3, 4, 2, 128, 16, [100, 260], BF, "slot")
    wide = torch.zeros((2, 3, 12, 128), dtype=BF)
    wide[:, :, 5:9] = d["q"]
    d["q"] = wide[:, :, 5:9]
    buf = torch.full((2, 4, 3, 128), 7.0, dtype=BF, device="cuda").transpose(1, 2)  # heads in front of tokens
    out = call(d, out=buf)
    assert out is buf
    check(d, out)


def test_another_stream():
    d = build(4, 3, 8, 2, 128, 16, [100, 260, 0, 1000], BF, "slot")
    want = call(d)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = call(d, stream=st)
    assert torch.equal(got, want)


def test_same_bits_every_time():
    d = build(6, 5, 8, 2, 128, 16, [1000, 260, 0, 3000, 77, 512], BF, "slot")
    first = call(d)
    for _ in range(3):
        assert torch.equal(call(d), first)


def test_graph_capture():
    import speculative_decoding_rejection_verify_gb300 as sv
    d = build(3, 4, 8, 2, 128, 16, [100, 1260, 0], BF, "slot")
    want = call(d)
    dev = {n: R.to_cuda(d[n]) for n in ("q", "k", "v")}
    pages, ctx = d["pages"].cuda(), torch.tensor(d["ctx"], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(want)
    ws = torch.zeros(sv.load().spec_paged_attention_workspace_bytes(3, 4, 8, 2, 128), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.paged_attention(dev["q"], dev["k"], dev["v"], pages, ctx, out=out, workspace_tensor=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_pool_beyond_32_bits():
    """Pages whose byte and element offsets pass 2^32."""
    import speculative_decoding_rejection_verify_gb300 as sv
    H, page, D, T = 8, 64, 128, 2
    num_pages = 2 ** 32 // (H * page * D) + 600  # elements past 2^32
    k = torch.empty((num_pages, page, H, D), dtype=BF, device="cuda")
    v = torch.empty_like(k)
    d = build(1, T, 16, H, D, page, [300], BF, "slot", garbage=False)
    n = d["pages"].shape[1]
    far = torch.tensor([[num_pages - 1 - 97 * i for i in range(n)]], dtype=torch.int32)
    for i in range(n):
        k[int(far[0, i])] = d["k"][int(d["pages"][0, i])].cuda()
        v[int(far[0, i])] = d["v"][int(d["pages"][0, i])].cuda()
    out = sv.paged_attention(d["q"].cuda(), k, v, far.cuda(), torch.tensor([300], dtype=torch.int32, device="cuda"))
    check(d, out)


def test_bad_device_data_stays_in_bounds():
    """Lengths outside the table are clamped and pages outside the pool read as zeros."""
    import speculative_decoding_rejection_verify_gb300 as sv
    d = build(3, 2, 4, 2, 64, 16, [40, 40, 40], BF, "slot", garbage=False)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    args = [R.to_cuda(d[n]) for n in ("q", "k", "v")]
    pages = d["pages"].clone()
    pages[1, 0] = -1
    pages[1, 1] = 2 ** 31 - 1
    out = sv.paged_attention(*args, pages.cuda(), i32([-5, 40, 2 ** 31 - 1]), i32([9, 2, 2]))
    assert torch.isfinite(out[:2]).all()
    d["ctx"][0] = 0  # a negative context counts as 0
    want, bound = R.attention(d["q"], d["k"], d["v"], d["pages"], d["ctx"], d["tb"], None, d["scale"])
    assert ((out.cpu().double() - want).abs() <= bound)[0].all()
    d["ctx"][1] = 40
    for i in (0, 1):  # as with pages of zeros
        d["k"][int(d["pages"][1, i])] = 0
        d["v"][int(d["pages"][1, i])] = 0
    want, bound = R.attention(d["q"], d["k"], d["v"], d["pages"], d["ctx"], d["tb"], None, d["scale"])
    assert ((out.cpu().double() - want).abs() <= bound)[1].all()
