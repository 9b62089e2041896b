"""spec_kv_append and spec_kv_keep against the formulas in float64."""
import math

import pytest
import torch

import _decode as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def table(n, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2).double() / rot)
    a = torch.arange(n).double()[:, None] * f
    return a.cos().float(), a.sin().float()


def run_append(B, T, Hq, H, D, page, ctx, dtype, layout, rot, interleaved, tb=None, positions=None, seed=1, packed=True,
               in_place=False):
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(seed)
    max_pages = -(-(max(ctx) + T) // page)
    num_pages = B * max_pages + 2
    k_pool, v_pool = R.pool(num_pages, page, H, D, dtype, layout, g)
    pages = R.tables(B, max_pages, num_pages, g)
    n = Hq + 2 * H
    qkv = (torch.randn((B, T, n, D), generator=g) * 2).to(BF)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:]
    if not packed:
        q, k, v = q.transpose(1, 2).contiguous().transpose(1, 2), k.contiguous(), v.contiguous()
    cos, sin = table(max(ctx) + T + 5, rot) if rot else (None, None)
    ks = vs = None
    if dtype == R.F8:
        ks, vs = torch.rand(H, generator=g) * 0.1 + 0.02, torch.rand(H, generator=g) * 0.1 + 0.002  # some overflow
    dev = [R.to_cuda(x) for x in (q, k, v, k_pool, v_pool)]
    flags = torch.zeros(B, dtype=torch.int32, device="cuda")
    out = sv.kv_append(*dev, pages.cuda(), i32(ctx), None if cos is None else cos.cuda(), None if sin is None else sin.cuda(),
                       None if tb is None else i32(tb), positions=None if positions is None else positions.cuda(),
                       interleaved=interleaved, k_scale=R.to_cuda(ks), v_scale=R.to_cuda(vs),
                       out=dev[0] if in_place else None, flags=flags)
    torch.cuda.synchronize()
    assert (flags == 0).all()
    tb = [T] * B if tb is None else tb
    raw = lambda c: (c.contiguous().view(torch.uint8) if dtype == R.F8 else c)  # noqa: E731
    got_k, got_v = dev[3].cpu(), dev[4].cpu()
    touched = torch.zeros((num_pages, page), dtype=torch.bool)
    for b in range(B):
        for t in range(T):
            if t >= tb[b]:
                assert out is None or (out[b, t] == 0).all()
                continue
            pos = ctx[b] + t if positions is None else int(positions[b, t])
            c, s = (cos[pos].double().tolist(), sin[pos].double().tolist()) if rot else ([], [])
            want, e = R.rotate(q[b, t].double(), c, s, interleaved)
            off = (out[b, t].cpu().double() - want).abs()
            assert (off <= R.U_BF16 * want.abs() + e).all()
            p, r = R.at(pages, b, ctx[b] + t, page)
            touched[p, r] = True
            want, e = R.rotate(k[b, t].double(), c, s, interleaved)
            for got, x, err, scale in ((got_k, want, e, ks), (got_v, v[b, t].double(), 0.0, vs)):
                entry = got[p, r].to(torch.float64)
                if dtype == R.F8:
                    x, err = x / scale.double()[:, None], err / scale.double()[:, None]
                    x = x.clamp(-448, 448)
                    # half a unit of 4 significant bits, 2^-10 below the normal range, and fp32's division
                    assert ((entry - x).abs() <= (x.abs() * U(R) + err) * (1 + 2.0 ** -20) + 2.0 ** -10).all()
                elif rot == 0 or got is got_v:
                    assert torch.equal(entry, x)
                else:
                    assert ((entry - x).abs() <= R.U_BF16 * x.abs() + err).all()
    for got, before in ((got_k, k_pool), (got_v, v_pool)):  # nothing else was written
        assert torch.equal(raw(got)[~touched].view(torch.uint8), raw(before)[~touched].view(torch.uint8))


def U(R):
    return R.U_E4M3


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, R.F8])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 128), (128, 32), (64, 16), (128, 0), (128, 48)])
def test_rotation_and_types(D, rot, dtype, interleaved):
    run_append(3, 4, 6, 2, D, 16, [0, 13, 700], dtype, "slot", rot, interleaved)


@pytest.mark.parametrize("B,T,Hq,H,page,layout", [(1, 1, 1, 1, 8, "slot"), (1, 1, 8, 8, 16, "head"), (2, 1, 7, 1, 32, "slot"),
                                                  (2, 70, 15, 5, 64, "head"), (5, 17, 64, 8, 16, "slot"), (1, 333, 4, 4, 256, "head")])
@pytest.mark.parametrize("dtype", [BF, R.F8])
def test_layouts(B, T, Hq, H, page, layout, dtype):
    run_append(B, T, Hq, H, 128, page, [11 * b for b in range(B)], dtype, layout, 128, False, seed=T)
    run_append(B, T, Hq, H, 64, page, [11 * b for b in range(B)], dtype, layout, 32, True, seed=T, packed=False)


def test_ragged_with_empty_requests():
    run_append(4, 6, 8, 2, 128, 16, [0, 100, 15, 3], BF, "slot", 128, False, tb=[0, 6, 3, 1])
    run_append(4, 6, 8, 2, 128, 16, [0, 100, 15, 3], R.F8, "head", 128, True, tb=[6, 0, 0, 5])


def test_positions_of_a_tree():
    ctx = [10, 0]
    depth = torch.tensor([0, 1, 2, 3, 1, 2, 3], dtype=torch.int32)
    run_append(2, 7, 4, 2, 64, 16, ctx, BF, "slot", 64, False,
               positions=torch.tensor(ctx, dtype=torch.int32)[:, None] + depth)


def test_in_place():
    run_append(2, 5, 8, 2, 128, 16, [3, 40], BF, "slot", 128, False, in_place=True)
    run_append(2, 5, 8, 2, 128, 16, [3, 40], BF, "slot", 64, True, in_place=True)


def test_keys_and_values_alone_and_special_values():
    import speculative_decoding_rejection_verify_gb300 as sv
    H, D, page = 2, 64, 16
    special = torch.tensor([0.0, -0.0, 1e30, -1e30, float("inf"), -float("inf"), float("nan"), 1e-30, 448.0, 464.0, 2.0 ** -10, 2.0 ** -9])
    x = special.repeat(D)[: H * D].view(1, 1, H, D).to(BF).cuda()
    for dtype in (BF, R.F8):
        k = torch.zeros((3, page, H, D), dtype=BF, device="cuda").to(dtype)
        v = torch.zeros((3, page, H, D), dtype=BF, device="cuda").to(dtype)
        assert sv.kv_append(None, x, x, k, v, i32([[2]]), i32([5])) is None
        want = x[0, 0].float().cpu()
        if dtype == R.F8:
            want = want.clamp(-448, 448).to(R.F8).float()
        for c in (k, v):
            got = c[2, 5].cpu().float()
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            assert torch.equal(got.nan_to_num(7.0), want.nan_to_num(7.0))


def test_bad_device_data_is_flagged_and_stays_in_bounds():
    import speculative_decoding_rejection_verify_gb300 as sv
    H, D, page, B, T = 2, 64, 16, 6, 3
    g = torch.Generator().manual_seed(2)
    k, v = [c.cuda() for c in R.pool(8, page, H, D, BF, "slot", g)]
    before = k.clone(), v.clone()
    x = torch.randn((B, T, H, D), generator=g).to(BF).cuda()
    cos, sin = (t.cuda() for t in table(40, 64))
    flags = torch.zeros(B, dtype=torch.int32, device="cuda")
    pages = i32([[0, 1], [-1, 2], [8, 2], [3, 4], [5, 6], [7, 7]])
    positions = i32([[0, 1, 2]] * 3 + [[39, 40, -1]] + [[0, 1, 2]] * 2)
    out = sv.kv_append(x, x, x, k, v, pages, i32([30, 0, 0, 0, -3, 2 ** 31 - 1]), cos, sin, i32([3, 3, 3, 3, 7, -1]),
                       positions=positions, flags=flags)
    torch.cuda.synchronize()
    assert flags.tolist() == [64, 64, 64, 128, 64 | 8, 8]
    assert torch.isfinite(out).all() and (out[5] == 0).all()
    assert torch.equal(k[2], before[0][2]) and torch.equal(v[7], before[1][7])
    assert torch.equal(v[1, 14:], x[0, :2]) and torch.equal(v[1, :14], before[1][1, :14])
    assert torch.equal(v[5, :3], x[4])  # a negative context counts as 0


@pytest.mark.parametrize("dtype", [BF, R.F8])
@pytest.mark.parametrize("layers,B,H,D,page,layout", [(None, 1, 1, 64, 8, "slot"), (1, 3, 2, 128, 16, "head"), (5, 4, 8, 128, 16, "slot"),
                                                      (3, 2, 5, 64, 64, "head")])
def test_keep(layers, B, H, D, page, layout, dtype):
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(4)
    T = 40
    ctx = [17 * b for b in range(B)]
    max_pages = -(-(max(ctx) + T) // page)
    num_pages = B * max_pages + 1
    k, v = R.pool(num_pages, page, H, D, dtype, layout, g, layers=layers)
    pages = R.tables(B, max_pages, num_pages, g)
    # paths that overlap their own targets, stand still, start late, or are empty
    paths = [[0, 5, 6, 7, 39], [1, 2, 3, 4, 5], [30, 31, 33, 38, 39], [0, 1, 2, 3, 4]]
    keep = [5, 4, 5, 0]
    path, n_keep = torch.tensor(paths[:B], dtype=torch.int32), torch.tensor(keep[:B], dtype=torch.int32)
    dev = [R.to_cuda(c) for c in (k, v)]
    sv.kv_keep(*dev, pages.cuda(), i32(ctx), path.cuda(), n_keep.cuda())
    torch.cuda.synchronize()
    for got, c in zip(dev, (k, v)):
        want = c.clone()
        w, s = (x.view(torch.uint8) if dtype == R.F8 else x for x in (want, c))
        for b in range(B):
            for i in range(keep[b]):
                to, fr = R.at(pages, b, ctx[b] + i, page), R.at(pages, b, ctx[b] + paths[b][i], page)
                w[..., to[0], to[1], :, :] = s[..., fr[0], fr[1], :, :]
        assert torch.equal(got.cpu().contiguous().view(torch.uint8), want.contiguous().view(torch.uint8))


def test_keep_leaves_bad_moves_out():
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(4)
    k, v = [c.cuda() for c in R.pool(4, 16, 1, 64, BF, "slot", g)]
    k0, v0 = k.clone(), v.clone()
    sv.kv_keep(k, v, i32([[0, 9], [1, 2]]), i32([10, 31]), i32([[1, 8, 30], [1, -4, 2 ** 31 - 1]]), i32([7, 3]))
    torch.cuda.synchronize()
    k0[0, 10] = k0[0, 11].clone()
    v0[0, 10] = v0[0, 11].clone()
    assert torch.equal(k, k0) and torch.equal(v, v0)


def test_append_then_keep_then_attend_sees_the_accepted_chain():
    """A tree's accepted chain, kept, is the same cache as that chain appended by itself."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(7)
    H, Hq, D, page, K, N, ctx = 2, 4, 64, 16, 3, 2, [14, 3]
    T = 1 + N * K
    k, v = [c.cuda() for c in R.pool(12, page, H, D, BF, "slot", g)]
    k2, v2 = k.clone(), v.clone()
    pages = R.tables(2, 3, 12, g).cuda()
    x = torch.randn((2, T, Hq + 2 * H, D), generator=g).to(BF).cuda()
    cos, sin = (t.cuda() for t in table(64, D))
    depth = i32([0] + [1, 2, 3] * N)
    split = lambda y: (y[:, :, :Hq], y[:, :, Hq:Hq + H], y[:, :, Hq + H:])  # noqa: E731
    sv.kv_append(*split(x), k, v, pages, i32(ctx), cos, sin, positions=(i32(ctx)[:, None] + depth).contiguous())
    chain = [1, 0]
    path = i32([[0] + [1 + c * K + j for j in range(K)] for c in chain])
    sv.kv_keep(k, v, pages, i32(ctx), path, i32([K + 1, K + 1]))
    alone = torch.stack([x[b, path[b].long()] for b in range(2)])
    sv.kv_append(*split(alone), k2, v2, pages, i32(ctx), cos, sin)
    for b in range(2):
        for s in range(ctx[b], ctx[b] + K + 1):
            p, r = R.at(pages.cpu(), b, s, page)
            assert torch.equal(k[p, r], k2[p, r]) and torch.equal(v[p, r], v2[p, r])
    assert math.isfinite(float(k.float().sum()))


def test_the_binding_refuses_what_does_not_fit():
    import speculative_decoding_rejection_verify_gb300 as sv
    dev = "cuda"
    c = torch.zeros((4, 16, 2, 64), dtype=BF, device=dev)
    pages, ctx = i32([[0, 1]]), i32([3])
    x = torch.zeros((1, 2, 2, 64), dtype=BF, device=dev)
    q = torch.zeros((1, 2, 4, 64), dtype=BF, device=dev)
    for bad in (lambda: sv.paged_attention(q.float(), c, c, pages, ctx), lambda: sv.paged_attention(q, c.half(), c.half(), pages, ctx),
                lambda: sv.paged_attention(q, c, c, pages.long(), ctx), lambda: sv.paged_attention(q, c, c, pages, ctx, mask=pages),
                lambda: sv.kv_append(q, x, x.float(), c, c, pages, ctx)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: sv.paged_attention(q, c, c[:3], pages, ctx), lambda: sv.paged_attention(q, c, c, pages, i32([1, 2])),
                lambda: sv.paged_attention(q[0], c, c, pages, ctx), lambda: sv.paged_attention(q, c, c, pages.cpu(), ctx),
                lambda: sv.paged_attention(q[..., :32], c, c, pages, ctx), lambda: sv.paged_attention(q, c[None], c[None], pages, ctx),
                lambda: sv.paged_attention(q.transpose(2, 3), c, c, pages, ctx), lambda: sv.kv_append(q, x, x[:, :1], c, c, pages, ctx),
                lambda: sv.kv_append(q, x, x, c, c, i32([[0], [1]]), ctx), lambda: sv.kv_append(q, x, x, c, c, pages, ctx, cos=ctx.float()),
                lambda: sv.kv_keep(c, c, pages, ctx, i32([0]), ctx), lambda: sv.kv_keep(c, c, pages, ctx, i32([[0], [1]]), ctx)):
        with pytest.raises(ValueError):
            bad()
    for bad, code in ((lambda: sv.paged_attention(q[:, :, :3], c, c, pages, ctx), 1),
                      (lambda: sv.paged_attention(q, c, c, pages, ctx, scale=float("nan")), 1),
                      (lambda: sv.paged_attention(q, c, c, pages, ctx, k_scale=torch.ones(2, device=dev)), 1),
                      (lambda: sv.paged_attention(q, c[:, :12], c[:, :12], pages, ctx), 2),
                      (lambda: sv.kv_append(None, x, x, c, c, pages, ctx, cos=torch.zeros((9, 4), device=dev), sin=torch.zeros((9, 4), device=dev)), 1)):
        with pytest.raises(sv.SpecVerifyError) as e:
            bad()
        assert e.value.code == code
