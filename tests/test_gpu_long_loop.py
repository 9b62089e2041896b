"""Decoding with drafts within a budget, through verdicts: what rejected drafts looked at must not count, for a chain of drafts (as the
documented loop has it) and for a tree."""
import math
import os
import re

import pytest
import torch

import _decode as R
import _pages as P

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_the_documented_loop_counts_accepted_tokens_only():
    """The block as users read it, one step with drafts that are rejected: weights are those of the accepted rows."""
    import speculative_decoding_rejection_verify_gb300 as sv
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = [b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "kv_weigh" in b]
    assert len(blocks) == 1
    g = torch.Generator().manual_seed(1)
    B, T, Hq, H, D, page, maxp, ctx, new = 3, 4, 8, 2, 64, 16, 8, [40, 0, 77], [1, 3, 4]
    num = B * maxp + 1
    k, v, ks, vs = P.pool(num, page, H, D, "slot", g)
    pages = R.tables(B, maxp, num, g)
    qkv = torch.randn((B, T, Hq + 2 * H, D), generator=g).to(BF).cuda()
    angle = torch.arange(200)[:, None] * torch.rand(D // 2, generator=g)
    weight, position = torch.rand((num, H, page), generator=g), torch.randint(0, 40, (num, H, page), generator=g).to(torch.int32)
    seen = [c + 9 for c in ctx]
    names = dict(sv=sv, q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + H], v=qkv[:, :, Hq + H:], k_cache=R.to_cuda(k), v_cache=R.to_cuda(v), ks=ks.cuda(),
                 vs=vs.cuda(), pages=pages.cuda(), ctx_len=i32(ctx), cos=angle.cos().cuda(), sin=angle.sin().cuda(), lse=torch.zeros((B, T, Hq), device="cuda"),
                 at=(i32(seen)[:, None] + torch.arange(T, dtype=torch.int32, device="cuda")).contiguous(), weight=weight.cuda(), position=position.cuda(),
                 new=i32(new), seen=i32(seen), budget=i32([1000] * B))  # nothing leaves
    at = names["at"].cpu()
    exec(blocks[0], names)
    torch.cuda.synchronize()
    assert names["ctx_len"].tolist() == [c + n for c, n in zip(ctx, new)] and int(names["moves"].abs().sum()) == 0
    keys = P.values(names["k_cache"].cpu(), names["ks"].cpu())
    want, want_p, bound = P.weigh(names["q"].cpu(), keys, pages, ctx, new, None, D ** -0.5, names["lse"].cpu(), weight, position, at, True)
    assert ((names["weight"].cpu().double() - want).abs() <= bound).all()
    assert torch.equal(names["position"].cpu(), want_p)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "pages"])
@pytest.mark.parametrize("N,K", [(1, 3), (3, 2)])
def test_rounds_of_drafts_within_a_budget(kind, N, K):
    """Append, attention, verdict, weigh, (keep,) select and move: after every round the weights are those that the accepted rows give,
    and at the end each head holds distinct positions, all of accepted tokens, the protected ones among them."""
    import speculative_decoding_rejection_verify_gb300 as sv
    g = torch.Generator().manual_seed(5)
    B, Hq, H, D, page, V, budget, first, recent = 2, 8, 2, 64, 16, 32, 40, 2, 12
    T = 1 + N * K
    maxp = 5
    num = B * maxp + 1
    pages = torch.randperm(num, generator=g)[:B * maxp].view(B, maxp).to(torch.int32)
    k, v = (torch.zeros((num, page, H, D), dtype=BF).to(BF if kind == "bf16" else R.F8).cuda() for _ in range(2))
    scales = {n: torch.ones((num, H), device="cuda") for n in ("k_scale", "v_scale")} if kind == "pages" else {}
    weight, position = torch.zeros((num, H, page), device="cuda"), torch.zeros((num, H, page), dtype=torch.int32, device="cuda")
    ctx, seen, dev_pages = i32([0, 0]), i32([0, 0]), pages.cuda()
    depth = torch.tensor([0] + [j + 1 for _ in range(N) for j in range(K)], dtype=torch.int32)
    bits = [1] + [1 | sum(1 << (1 + n * K + i) for i in range(j + 1)) for n in range(N) for j in range(K)]
    mask = torch.tensor(bits, dtype=torch.int64).expand(B, T).contiguous()
    accepted = [[] for _ in range(B)]  # every position's key and value
    rejected = 0
    for _ in range(25):
        qkv = torch.randn((B, T, Hq + 2 * H, D), generator=g).to(BF)
        q, kk, vv = (x.contiguous() for x in (qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H], qkv[:, :, Hq + H:]))
        at = (seen.cpu()[:, None] + depth).to(torch.int32).contiguous()
        qr = sv.kv_append(q.cuda(), kk.cuda(), vv.cuda(), k, v, dev_pages, ctx, **scales)
        lse = torch.zeros((B, T, Hq), device="cuda")
        sv.paged_attention(qr, k, v, dev_pages, ctx, mask=mask.cuda(), lse=lse, **scales)
        p, dq = torch.randn((B, N, K + 1, V), generator=g).cuda(), torch.randn((B, N, K, V), generator=g).cuda()
        draft = torch.randint(0, V, (B, N, K), generator=g).to(torch.int32).cuda()
        u, r = torch.rand((B, N, K), generator=g).cuda(), torch.rand(B, generator=g).cuda()
        if N == 1:
            _, n_acc, _ = sv.verify(p[:, 0].contiguous(), dq[:, 0].contiguous(), draft[:, 0].contiguous(), None, u[:, 0].contiguous(), r)
            chain = torch.zeros_like(n_acc)
        else:
            _, n_acc, chain, _ = sv.verify_multi(p, dq, draft, u, r, draft_temperature=1.0)
        kept = n_acc + 1
        path = torch.cat([torch.zeros((B, 1), dtype=torch.int32, device="cuda"),
                          1 + chain.clamp(min=0)[:, None] * K + torch.arange(K, dtype=torch.int32, device="cuda")], 1).contiguous()
        n, c, branch = kept.tolist(), ctx.tolist(), path.tolist()
        before, before_p = weight.cpu(), position.cpu()
        keys = P.values(k.cpu(), scales["k_scale"].cpu()) if scales else k.cpu().to(torch.float64)
        if N == 1:
            sv.kv_weigh(qr, k, dev_pages, ctx, lse, weight, position, t_per_row=kept, positions=at.cuda(), k_scale=scales.get("k_scale"))
            want, want_p, bound = P.weigh(q, keys, pages, c, n, None, D ** -0.5, lse.cpu(), before, before_p, at, kind != "bf16")
        else:
            out = torch.ones((B, T), dtype=torch.bool)
            for b in range(B):
                out[b, branch[b][:n[b]]] = False
            lse.masked_fill_(out.cuda()[..., None], math.inf)
            sv.kv_weigh(qr, k, dev_pages, ctx, lse, weight, position, mask=mask.cuda(), positions=at.cuda(), k_scale=scales.get("k_scale"))
            sv.kv_keep(k, v, dev_pages, ctx, path, kept, weight=weight, position=position, **scales)
            want, want_p, bound = P.weigh(q, keys, pages, c, [T] * B, mask, D ** -0.5, lse.cpu(), before, before_p, at, kind != "bf16")
            for b in range(B):
                for i, t in enumerate(branch[b][:n[b]]):
                    to, of = R.at(pages, b, c[b] + i, page), R.at(pages, b, c[b] + t, page)
                    for x in (want, want_p, bound):
                        x[to[0], :, to[1]] = x[of[0], :, of[1]]
        assert ((weight.cpu().double() - want).abs() <= bound).all() and torch.equal(position.cpu(), want_p)
        for b in range(B):
            accepted[b] += [(kk[b, t].double(), vv[b, t].double()) for t in branch[b][:n[b]]]
            rejected += T - n[b]
        ctx, seen = ctx + kept, seen + kept
        if int(ctx.max()) > budget + 16:
            source, target, moves, ctx = sv.kv_select(weight, position, dev_pages, ctx, i32([budget] * B), seen=seen, first=first, recent=recent)
            sv.kv_move(k, v, dev_pages, ctx, source, target, moves, weight=weight, position=position, **scales)
    torch.cuda.synchronize()
    assert rejected > 25
    deq = [P.values(x.cpu(), s.cpu()) if scales else x.cpu().to(torch.float64) for x, s in zip((k, v), scales.values() or (0, 0))]
    for b in range(B):
        m, total = int(ctx[b]), int(seen[b])
        assert total == len(accepted[b]) and m <= total
        slots = torch.arange(m)
        pg, row = pages[b].long()[slots // page], slots % page
        for h in range(H):
            held = position.cpu()[pg, h, row].tolist()
            assert len(set(held)) == m and max(held) < total
            assert set(range(first)) <= set(held) and set(range(max(total - recent, 0), total)) <= set(held)
            for side, entry in enumerate(deq):
                want = torch.stack([accepted[b][i][side][h] for i in held])
                # E4M3: half a step, 2^-4 of the value or 2^-10 of its (page's) scale, which is 2^-6 at most here, each of a few times that it grows
                tol = 0.0 if kind == "bf16" else 2.0 ** -4 * want.abs() + (2.0 ** -10 if kind == "e4m3" else 8 * 2.0 ** -10 * 2.0 ** -6)
                assert ((entry[pg, row, h] - want).abs() <= tol).all()
