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
    """Of items that one block takes whole (the narrow table) and of those that are cut and joined: a row and its sum come out as
    they are, or both as NaN."""
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
    lost = torch.isnan(out).any(-1)
    assert lost.any() and torch.equal(torch.isnan(lse), lost)
    assert torch.equal(out[~lost], want[~lost]) and torch.equal(lse[~lost], sums[~lost])
    again, sums2 = call()
    assert torch.equal(again, want) and torch.equal(sums2, sums)
