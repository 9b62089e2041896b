"""The decode-step operators where their rules meet their limits: weights at a rounding boundary, sizes at which
another variant or another round of a loop begins, and calls that are captured or made on several streams."""
import pytest
import torch

import _decode as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def attention_inputs(B, ctx, seed, Hq=8, H=2, D=128, page=16, T=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    pages = -(-(ctx + T) // page)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(BF)  # noqa: E731
    return [rand(B, T, Hq, D), rand(B * pages, page, H, D), rand(B * pages, page, H, D),
            torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages), i32([ctx] * B)]


# ------------------------------------------------------------------------------------------------
# paged_attention
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("Hq", [1, 16, 32, 64, 80, 128])
@pytest.mark.parametrize("dtype", [BF, R.F8])
def test_equal_values_come_back_as_they_are(Hq, dtype):
    """The weights of a row sum to 1, whatever each is rounded to: with one value in every slot the output is that
    value.  Slot 200's score passes the maximum of the first tile by up to 7.8 in log2 units, so its weight is not a
    power of two and outweighs all others together.  (fp32 sums of 300 terms are off by 300 * 2^-24, far inside
    half a unit of the output's 8 bits.)"""
    import speculative_decoding_rejection_verify_gb300 as sv
    D, page, ctx = 64, 16, 299
    k = torch.zeros((19, page, 1, D))
    k.view(-1, D)[:, 0] = -64.0
    k.view(-1, D)[0, 0] = 0.0
    k.view(-1, D)[200, 0] = 1.0
    v = torch.full((19, page, 1, D), 1.875)
    q = torch.zeros((1, 1, Hq, D), dtype=BF)
    q[0, 0, :, 0] = torch.linspace(5.4, 0.3, Hq).to(BF)
    out = sv.paged_attention(q.cuda(), k.to(dtype).cuda(), v.to(dtype).cuda(), torch.arange(19, dtype=torch.int32, device="cuda")[None],
                             i32([ctx]), scale=1.0)
    assert (out == 1.875).all()


@pytest.mark.parametrize("Hq,D", [(4, 128), (64, 64)])
def test_a_query_with_one_large_element_over_e4m3(Hq, D):
    """Queries enter an E4M3 cache's scores as two E4M3 numbers: exactly where an element reaches 2^-9 of its row's largest, and
    to 2^-17 of that largest elsewhere.  Here the largest meets zeros, so the scores are all made of the others."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(9)
    T, ctx, page, scale = 2, 250, 16, D ** -0.5
    q = torch.randn((1, T, Hq, D), generator=g)
    q[..., 0] = 700.0
    q[:, 1] *= 1e-3
    q = q.to(BF)
    k, v = R.pool(16, page, 1, D, R.F8, "slot", g)
    k.view(torch.uint8)[..., 0] = 0
    pages = torch.arange(16, dtype=torch.int32)[None]
    got = sv.paged_attention(q.cuda(), k.cuda(), v.cuda(), pages.cuda(), i32([ctx])).cpu().double()
    want, bound = R.attention(q, k, v, pages, [ctx], [T], None, scale)
    size, _ = R.attention(q, k, v.float().abs().to(R.F8), pages, [ctx], [T], None, scale)
    # a score is off by 2^-17 of the row's largest times the sum of a key's elements, a normalised weight by twice that
    off = 2.0 ** -17 * q.double().abs().amax(-1, keepdim=True) * k.double().abs().sum(-1).max() * scale
    assert ((got - want).abs() <= bound + (torch.exp(2 * off) - 1) * size).all()
    # elements within 2^-9 of the largest: no further error
    q[..., 0] = 300.0
    q[..., 1:] = (q[..., 1:].float().sign() * (0.6 + torch.rand(q[..., 1:].shape, generator=g) * 0.4)).to(BF)
    got = sv.paged_attention(q.cuda(), k.cuda(), v.cuda(), pages.cuda(), i32([ctx])).cpu().double()
    want, bound = R.attention(q, k, v, pages, [ctx], [T], None, scale)
    assert ((got - want).abs() <= bound).all()


@pytest.mark.parametrize("T,Hq", [(1, 4), (4, 16), (17, 8), (16, 16), (64, 8)])
@pytest.mark.parametrize("ctx,width", [(300, 0), (1500, 0), (300, 4000)])
@pytest.mark.parametrize("dtype", [BF, R.F8])
def test_a_wait_that_runs_out_ends_the_call_with_nan_rows(T, Hq, ctx, width, dtype):
    """Every wait inside the kernel gives up after one try, with copies in flight: the call ends, all rows say so, and
    the next call is exact."""
    import speculative_decoding_rejection_verify_gb300 as sv
    q, k, v, pages, n = attention_inputs(3, ctx, 5, Hq=Hq, T=T)
    k, v = k.to(dtype), v.to(dtype)
    if width:
        pages = torch.cat([pages, i32([[0] * width] * 3)], 1).contiguous()
    want = sv.paged_attention(q, k, v, pages, n)
    sv.set_test_hooks(2)
    try:
        lost = sv.paged_attention(q, k, v, pages, n)
        torch.cuda.synchronize()
    finally:
        sv.set_test_hooks(0)
    assert torch.isfinite(want).all() and torch.isnan(lost).all()
    assert torch.equal(sv.paged_attention(q, k, v, pages, n), want)


# ------------------------------------------------------------------------------------------------
# kv_append
# ------------------------------------------------------------------------------------------------
def test_entries_are_the_quotients_codes():
    """An E4M3 entry is x / scale in fp32, rounded once: the code of the exact quotient where that lies halfway between two
    codes (odd multiples of 5 bits times a scale of few bits), 0 / scale = 0 however small the scale is."""
    import speculative_decoding_rejection_verify_gb300 as sv
    D, page = 64, 16
    scales = [3.0, 5.0, 7.0, 0.0390625, 1.75, 0.1, 0.4375, 7 * 2.0 ** -120, 3 * 2.0 ** -149, 2.0 ** -140, 7 * 2.0 ** 120, 2.0 ** 127]
    H = len(scales)
    ties = torch.tensor([17.0, 19, 21, 23, 25, 27, 29, 31])
    x = torch.zeros((1, 1, H, D))
    for h, s in enumerate(scales):
        x[0, 0, h, :8] = ties * s
        x[0, 0, h, 8:16] = -ties * s / 16
        x[0, 0, h, 16:48] = torch.randn(32, generator=torch.Generator().manual_seed(h)) * s * 30
        x[0, 0, h, 48:56] = torch.tensor([1e38, -1e38, float("inf"), -float("inf"), 1e-38, 1.0, -3.0, 2.0 ** -130])
    x = x.to(BF)
    scale = torch.tensor(scales)
    want = (x[0, 0].float() / scale[:, None]).clamp(-448, 448).to(R.F8).float()
    k = torch.zeros((1, page, H, D), device="cuda").to(R.F8)
    v = torch.zeros((1, page, H, D), device="cuda").to(R.F8)
    sv.kv_append(None, x.cuda(), x.cuda(), k, v, i32([[0]]), i32([3]), k_scale=scale.cuda(), v_scale=scale.cuda())
    for c in (k, v):
        assert torch.equal(c[0, 3].float().cpu(), want)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF, R.F8])
@pytest.mark.parametrize("D,rot,Hq,H", [(128, 128, 8, 2), (128, 48, 5, 1), (64, 64, 7, 7), (64, 32, 2, 1), (128, 0, 3, 3)])
def test_append_of_thousands_of_tokens(D, rot, Hq, H, dtype, interleaved):
    """From 16 tokens per SM on a token has 64 threads: 48 rotated elements leave some of them without a unit, and a token's
    heads take several rounds."""
    import speculative_decoding_rejection_verify_gb300 as sv
    B, page, ctx, tb = 2, 32, [7, 100], [1700, 1733]
    T = max(tb)
    assert B * T >= 16 * torch.cuda.get_device_properties(0).multi_processor_count
    g = torch.Generator().manual_seed(D + rot)
    max_pages = -(-(max(ctx) + T) // page)
    k, v = R.pool(B * max_pages, page, H, D, dtype, "head", g)
    pages = R.tables(B, max_pages, B * max_pages, g)
    x = (torch.randn((B, T, Hq + 2 * H, D), generator=g) * 2).to(BF)
    f = 10000.0 ** (-torch.arange(0, max(rot, 2), 2).double() / max(rot, 1))
    a = torch.arange(max(ctx) + T).double()[:, None] * f
    cos, sin = (a.cos().float(), a.sin().float()) if rot else (None, None)
    scales = [torch.rand(H, generator=g) * 0.1 + 0.02 for _ in range(2)] if dtype == R.F8 else [None, None]
    dev, kc, vc = x.cuda(), R.to_cuda(k), R.to_cuda(v)
    out = sv.kv_append(dev[:, :, :Hq], dev[:, :, Hq:Hq + H], dev[:, :, Hq + H:], kc, vc, pages.cuda(), i32(ctx),
                       None if cos is None else cos.cuda(), None if sin is None else sin.cuda(), i32(tb), interleaved=interleaved,
                       k_scale=R.to_cuda(scales[0]), v_scale=R.to_cuda(scales[1])).cpu().double()
    for b in range(B):
        n = tb[b]
        slot = ctx[b] + torch.arange(n)
        y, err = x[b, :n].double(), torch.zeros((n, Hq + 2 * H, D), dtype=torch.float64)
        if rot:
            one, two = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
            c, s = cos[slot].double()[:, None], sin[slot].double()[:, None]
            p, q = y[:, :Hq + H, one].clone(), y[:, :Hq + H, two].clone()
            y[:, :Hq + H, one], y[:, :Hq + H, two] = p * c - q * s, q * c + p * s
            err[:, :Hq + H, one] = err[:, :Hq + H, two] = 2.0 ** -22 * (p.abs() + q.abs())
        assert ((out[b, :n] - y[:, :Hq]).abs() <= R.U_BF16 * y[:, :Hq].abs() + err[:, :Hq]).all() and (out[b, n:] == 0).all()
        at = pages[b].long()[slot // page], slot % page
        for got, scale, h0 in ((kc, scales[0], Hq), (vc, scales[1], Hq + H)):
            raw = got.cpu()
            entry = raw.view(torch.uint8)[at].view(R.F8).double() if dtype == R.F8 else raw[at].double()
            want, e = y[:, h0:h0 + H], err[:, h0:h0 + H]
            if dtype == R.F8:
                want, e = (want / scale.double()[:, None]).clamp(-448, 448), e / scale.double()[:, None]
                assert ((entry - want).abs() <= (want.abs() * R.U_E4M3 + e) * (1 + 2.0 ** -20) + 2.0 ** -10).all()
            else:
                assert ((entry - want).abs() <= R.U_BF16 * want.abs() + e).all()


# ------------------------------------------------------------------------------------------------
# kv_keep
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, R.F8])
@pytest.mark.parametrize("layers", [1, 3])
def test_keep_of_many_entries(layers, dtype):
    """More kept entries than a warp's lanes (32) and than a round's moves (64), with moves that begin, end and stand
    still on both sides of these."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(6)
    most, page, H, D = 150, 16, 2, 64
    paths = [[i + 1 for i in range(most)], [i if i < 31 else i + 2 for i in range(most)], [i if i < 64 else 2 * i - 63 for i in range(most)],
             [2 * i for i in range(most)], [i if i % 3 == 0 and i < 60 else i + (1 if i < 61 else 7) for i in range(most)],
             [i + 40 for i in range(most)]]
    paths[4] = sorted(set(paths[4]))
    paths[4] += [paths[4][-1] + 1 + i for i in range(most - len(paths[4]))]
    keep = [150, 97, 150, 65, 128, 64]
    for p in paths:
        assert len(p) == most and all(b > a for a, b in zip(p, p[1:]))
    ctx = [0, 5, 16, 31, 100, 2]
    B = len(paths)
    max_pages = -(-(max(ctx) + max(max(p) for p in paths) + 1) // page)
    k, v = R.pool(B * max_pages, page, H, D, dtype, "slot", g, layers=layers)
    pages = R.tables(B, max_pages, B * max_pages, g)
    dev = [R.to_cuda(c) for c in (k, v)]
    sv.kv_keep(*dev, pages.cuda(), i32(ctx), i32(paths), i32(keep))
    for got, c in zip(dev, (k, v)):
        s = c.view(torch.uint8) if dtype == R.F8 else c
        w = s.clone()
        for b in range(B):
            for i in range(keep[b]):
                to, fr = R.at(pages, b, ctx[b] + i, page), R.at(pages, b, ctx[b] + paths[b][i], page)
                w[:, to[0], to[1]] = s[:, fr[0], fr[1]]
        raw = got.cpu()
        assert torch.equal(raw.view(torch.uint8) if dtype == R.F8 else raw, w)


# ------------------------------------------------------------------------------------------------
# process_logits
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("B,V", [(610, 9001), (420, 9001), (420, 9008), (610, 9008)])
@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_longer_stretches_of_the_vocabulary(B, V, dtype):
    """Batches that take 4096 and 8192 tokens a block, with rows on 16-byte boundaries and on any."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    want = 8192 if B == 610 else 4096
    assert next(s for s in (8192, 4096, 2048) if B * -(-V // s) >= 8 * sms) == want
    from test_gpu_logits import build, check
    z, r = build(B, 2, V, V + B, bias=20)
    check(z, r, dtype, in_place=V % 2 == 1)


@pytest.mark.parametrize("V", [2048, 2051])
def test_repeated_tokens_logits_are_quotients(V):
    """z / repetition is the quotient rounded to fp32, wherever the row begins."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(5)
    B, T = 6, 3
    z = torch.randn((B, T, V), generator=g) * 10
    z[:, :, :200] = z[:, :, :200].abs() * torch.exp(torch.randn(200, generator=g) * 10)
    rep = torch.tensor([1.1, 1.0 / 3, 1.9999999, 1.3, 7.0, 0.7])
    ids = torch.arange(V, dtype=torch.int32).expand(B, V).contiguous()
    n = torch.full((B,), V, dtype=torch.int32)
    got = sv.process_logits(z.cuda(), history=ids.cuda(), history_len=n.cuda(), prompt_len=n.cuda(), repetition=rep.cuda()).cpu()
    r = rep[:, None, None]
    assert torch.equal(got, torch.where(z > 0, z / r, z * r))


# ------------------------------------------------------------------------------------------------
# captured calls and their scratch
# ------------------------------------------------------------------------------------------------
def test_a_captured_call_without_a_workspace_keeps_its_memory():
    """Captured behind a warm call, then a larger call on the same stream, fresh tensors, replays: the result is right
    and nothing else changes."""
    import speculative_decoding_rejection_verify_gb300 as sv
    small, large = attention_inputs(2, 1500, 1), attention_inputs(2, 1500, 2, Hq=64, T=16)
    want = sv.paged_attention(*small)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        sv.paged_attention(*small)
    st.synchronize()
    out = torch.zeros_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        sv.paged_attention(*small, out=out)
    with torch.cuda.stream(st):
        sv.paged_attention(*large)
        fresh = [torch.full((1 << 18,), 7.0, device="cuda") for _ in range(64)]
        for _ in range(3):
            out.zero_()
            graph.replay()
            st.synchronize()
            assert torch.equal(out, want)
    assert all((x == 7.0).all() for x in fresh)


def test_two_graphs_of_one_stream_replay_beside_each_other():
    import speculative_decoding_rejection_verify_gb300 as sv
    inputs = [attention_inputs(2, 3000, seed) for seed in (1, 2)]
    want = [sv.paged_attention(*x) for x in inputs]
    torch.cuda.synchronize()
    outs, graphs, streams = [torch.zeros_like(w) for w in want], [], [torch.cuda.Stream() for _ in range(2)]
    for x, out in zip(inputs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=streams[0]):
            for _ in range(20):
                sv.paged_attention(*x, out=out)
    for _ in range(5):
        for out, graph, st in zip(outs, graphs, streams):
            with torch.cuda.stream(st):
                out.zero_()
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, w) for out, w in zip(outs, want))


def test_a_captured_verify_without_a_workspace():
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator(device="cuda").manual_seed(3)
    B, K, V = 6, 3, 5000
    rand = lambda *shape: torch.rand(shape, generator=g, device="cuda")  # noqa: E731
    p, q = rand(B, K + 1, V) * 4, rand(B, K, V) * 4
    draft = torch.randint(0, V, (B, K), generator=g, device="cuda", dtype=torch.int32)
    args = (p, q, draft, None, rand(B, K), rand(B))
    want = sv.verify(*args)[:2]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        sv.verify(*args)
    st.synchronize()
    out = [torch.zeros_like(w) for w in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        sv.verify(*args, out=tuple(out))
    with torch.cuda.stream(st):
        sv.sample(rand(600, 40000), rand(600))  # a larger scratch on the same stream
        fresh = [torch.full((1 << 16,), 7.0, device="cuda") for _ in range(64)]
        graph.replay()
        st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want)) and all((x == 7.0).all() for x in fresh)


# ------------------------------------------------------------------------------------------------
# the device
# ------------------------------------------------------------------------------------------------
def test_calls_refuse_tensors_that_are_not_on_the_current_device(monkeypatch):
    """With a stand-in for the current device's number nothing is launched, and every entry point says so."""
    import speculative_decoding_rejection_verify_gb300 as sv
    q, k, v, pages, ctx = attention_inputs(1, 40, 1)
    p = torch.zeros((1, 2, 64), device="cuda")
    one, key = i32([[0]]), k[:3].unsqueeze(0)
    before = k.clone()
    calls = [lambda: sv.paged_attention(q, k, v, pages, ctx), lambda: sv.kv_append(q, key[:, :, 0], key[:, :, 1], k, v, pages, ctx),
             lambda: sv.kv_keep(k, v, pages, ctx, one, ctx), lambda: sv.process_logits(p),
             lambda: sv.verify(p, None, one, temperature=0.0), lambda: sv.sample(p[0], temperature=0.0),
             lambda: sv.verify_multi(p[None], None, one[None], temperature=0.0)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    before = k.clone()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(sv.decode, "_current_device", lambda: 1)
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()
    with pytest.raises(ValueError, match="current device"):
        sv.verify_host(p.cpu().numpy(), None, one.cpu().numpy(), temperature=0.0, device="cuda:0")
    monkeypatch.undo()
    torch.cuda.synchronize()
    assert torch.equal(k, before)


# ------------------------------------------------------------------------------------------------
# refusals
# ------------------------------------------------------------------------------------------------
def test_sizes_beyond_the_limits_are_unsupported():
    """The binding raises what the library says of the sizes: 2 beyond a limit, 1 where they cannot be."""
    import speculative_decoding_rejection_verify_gb300 as sv

    def code(T=2, Hq=4, H=2, D=64):
        c = torch.zeros((3, 16, H, D), dtype=BF, device="cuda")
        q = torch.zeros((1, T, Hq, D), dtype=BF, device="cuda")
        with pytest.raises(sv.SpecVerifyError) as e:
            sv.paged_attention(q, c, c, i32([[0, 1, 2]]), i32([3]))
        return e.value.code

    assert code(T=65) == 2
    assert code(D=96) == 2
    assert code(Hq=129, H=1) == 2
    assert code(Hq=3) == 1


def test_a_workspace_on_the_host_is_refused():
    import speculative_decoding_rejection_verify_gb300 as sv
    ws = torch.zeros(64 << 20, dtype=torch.uint8)
    p, draft = torch.zeros((1, 2, 64), device="cuda"), i32([[0]])
    for call in (lambda w: sv.paged_attention(*attention_inputs(1, 20, 1), workspace_tensor=w),
                 lambda w: sv.verify(p, None, draft, temperature=0.0, workspace_tensor=w),
                 lambda w: sv.sample(p[0], temperature=0.0, workspace_tensor=w),
                 lambda w: sv.verify_multi(p[None], None, draft[None], temperature=0.0, workspace_tensor=w)):
        with pytest.raises(ValueError):
            call(ws)
        with pytest.raises(TypeError):
            call(ws.cuda().view(torch.int32))
        call(ws.cuda())
    with pytest.raises(ValueError):
        sv.verify_host(p.cpu().numpy(), None, draft.cpu().numpy(), temperature=0.0, staging=ws)


def test_halves_of_a_pair_are_refused():
    """bias without its ids and sin without cos were left out of the result without a word."""
    import speculative_decoding_rejection_verify_gb300 as sv
    z = torch.zeros((2, 1, 64), device="cuda")
    with pytest.raises(ValueError, match="bias"):
        sv.process_logits(z, bias=torch.ones((2, 64), device="cuda"))
    q, k, v, pages, ctx = attention_inputs(1, 40, 1)
    x = torch.zeros((1, 3, 2, 128), dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="sin"):
        sv.kv_append(q, x, x, k, v, pages, ctx, sin=torch.zeros((64, 32), device="cuda"))


def test_no_position_at_all_with_drafts():
    import speculative_decoding_rejection_verify_gb300 as sv
    z = torch.zeros((2, 0, 64), device="cuda")
    assert sv.process_logits(z, draft=torch.zeros((2, 0), dtype=torch.int32, device="cuda")).shape == z.shape


def test_queries_turn_by_their_position_also_without_a_slot():
    """A context longer than the page table: the entries have no slot (flagged), the queries still are at ctx_len + t."""
    import speculative_decoding_rejection_verify_gb300 as sv
    q, k, v, pages, _ = attention_inputs(2, 40, 1)
    x = torch.zeros((2, 3, 2, 128), dtype=BF, device="cuda")
    angle = torch.arange(400, device="cuda").double()[:, None] * 10000.0 ** (-torch.arange(64, device="cuda").double() / 64)
    cos, sin = angle.cos().float(), angle.sin().float()
    flags, ctx = i32([0, 0]), i32([300, 46])  # the table holds 48 slots
    before = k.clone()
    out = sv.kv_append(q, x, x, k, v, pages, ctx, cos, sin, flags=flags)
    want = sv.kv_append(q, x, x, k.clone(), v.clone(), pages, i32([0, 0]), cos, sin, positions=i32([[300, 301, 302], [46, 47, 48]]))
    assert torch.equal(out, want) and flags.tolist() == [64, 64]
    changed = (k != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert changed == [int(pages[1, 2])]
    flags.zero_()
    sv.kv_append(q, x, x, k, v, pages, i32([2 ** 31 - 1, 0]), cos, sin, flags=flags)  # no position that large
    assert flags.tolist() == [64 | 128, 0]
