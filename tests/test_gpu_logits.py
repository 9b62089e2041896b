"""spec_process_logits against the formula in float64 (the bound is six fp32 roundings of the terms' sizes,
and the output's own rounding)."""
import numpy as np
import pytest
import torch

import _decode as R

pytestmark = pytest.mark.gpu


def build(B, T, V, seed, L=50, bias=5, mask=True, penalties=True, spread=None):
    g = np.random.default_rng(seed)
    r = {}
    hot = g.integers(0, V, max(2, min(V, 12)))
    r["history"] = np.where(g.random((B, L)) < 0.7, g.choice(hot, (B, L)), g.integers(0, V, (B, L))).astype(np.int32)
    r["history_len"] = g.integers(0, L + 1, B).astype(np.int32)
    r["prompt_len"] = (r["history_len"] // 2).astype(np.int32)
    r["draft"] = g.choice(hot, (B, T - 1)).astype(np.int32)
    if penalties:
        r["repetition"] = (g.random(B) * 1.5 + 0.5).astype(np.float32)
        r["presence"] = (g.random(B) * 2 - 1).astype(np.float32)
        r["frequency"] = g.random(B).astype(np.float32)
    if bias:
        r["bias_ids"] = np.stack([g.permutation(V)[:bias] for _ in range(B)]).astype(np.int32)
        r["bias"] = g.normal(0, 3, (B, r["bias_ids"].shape[1])).astype(np.float32)
    if mask:
        m = g.integers(-2 ** 31, 2 ** 31, (B, T, (V + 31) // 32))
        r["mask"] = (m if spread is None else m & spread).astype(np.int32)
    z = torch.from_numpy(g.normal(0, 4, (B, T, V)).astype(np.float32))
    return z, r


def call(z, r, **kw):
    import speculative_decoding_rejection_verify_gb300 as sv
    out = sv.process_logits(z, **{k: torch.from_numpy(np.ascontiguousarray(x)).cuda() for k, x in r.items()}, **kw)
    torch.cuda.synchronize()
    return out


def check(z, r, dtype, tb=None, in_place=False):
    B, T, V = z.shape
    z = z.to(dtype)
    dev = z.cuda()
    out = dev if in_place else torch.full(z.shape, 123.0, dtype=dtype, device="cuda")
    if tb is not None:
        r = dict(r, t_per_row=np.array(tb, np.int32))
    got = call(dev, r, out=out).cpu().double().numpy()
    tb = [T] * B if tb is None else tb
    want, bound = R.logits(z.float().numpy(), r, tb)
    for b in range(B):
        same = z[b, tb[b]:].double().numpy() if in_place else 123.0
        assert (got[b, tb[b]:] == same).all()
        w, g, e = want[b, :tb[b]], got[b, :tb[b]], bound[b, :tb[b]]
        assert (np.isneginf(w) == np.isneginf(g)).all()
        fine = np.isfinite(w)
        w, g, e = w[fine], g[fine], e[fine]
        e = e + (R.U_BF16 if dtype == torch.bfloat16 else R.U_F32) * np.abs(w)
        assert (np.abs(g - w) <= e).all(), np.abs(g - w).max()


DT = [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("V", [1, 3, 8, 31, 32, 33, 1000, 1001, 2047, 2048, 8184, 8192, 8200, 16385, 32000, 50257])
def test_vocabulary_sizes(V, dtype):
    check(*build(2, 3, V, V, bias=min(V, 5)), dtype)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,T", [(1, 1), (1, 17), (7, 2), (40, 5), (3, 64)])
def test_batches(B, T, dtype):
    check(*build(B, T, 4104, B), dtype)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("parts", [dict(mask=False), dict(bias=0), dict(penalties=False), dict(mask=False, bias=0),
                                   dict(mask=False, bias=0, penalties=False), dict(L=1), dict(L=5000), dict(bias=300)])
def test_parts_alone(parts, dtype):
    check(*build(3, 4, 10000, 5, **parts), dtype)


@pytest.mark.parametrize("dtype", DT)
def test_ragged_and_in_place(dtype):
    z, r = build(5, 6, 9008, 11)
    check(z, r, dtype, tb=[0, 6, 1, 3, 5])
    check(z, r, dtype, tb=[2, 0, 6, 6, 1], in_place=True)
    check(z[:, :, :9005].contiguous(), dict(r, **build(5, 6, 9005, 12)[1]), dtype, tb=[2, 0, 6, 6, 1], in_place=True)


@pytest.mark.parametrize("dtype", DT)
def test_a_mask_that_allows_nothing_or_all(dtype):
    z, r = build(2, 3, 2056, 3)
    r["mask"][0, 1] = 0
    r["mask"][1, 2] = -1
    check(z, r, dtype)
    assert torch.isneginf(call(z.to(dtype).cuda(), r)[0, 1]).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("V", [2056, 2057])
def test_special_logits(dtype, V):
    """Infinities and NaN stay where they are allowed, and are -inf where they are not."""
    z, r = build(1, 2, V, 3, penalties=False, bias=0)
    low = torch.finfo(dtype).min
    z[0, 0, :6] = torch.tensor([float("nan"), float("inf"), -float("inf"), low, 0.0, -0.0])
    z[0, 1, :6] = z[0, 0, :6]
    r["mask"][0, 0] = 0
    r["mask"][0, 1] = -1
    got = call(z.to(dtype).cuda(), r).cpu()
    assert torch.isneginf(got[0, 0]).all()
    assert torch.equal(got[0, 1].nan_to_num(3.0, 4.0, 5.0), z[0, 1].to(dtype).nan_to_num(3.0, 4.0, 5.0))


def test_ids_outside_the_vocabulary_are_skipped():
    z, r = build(2, 4, 777, 8)
    r["history"][:, ::5] = -1
    r["history"][:, 1::5] = 777
    r["history"][:, 2::7] = 2 ** 31 - 1
    r["draft"][:, 1] = -2 ** 31
    r["bias_ids"][:, 0] = -3
    r["bias_ids"][:, 1] = 777
    check(z, r, torch.float32)
    r["history_len"] = np.array([-4, 10 ** 9], np.int32)
    r["prompt_len"] = np.array([5, -1], np.int32)
    check(z, r, torch.float32)


def test_the_later_of_two_bias_entries_holds():
    z, r = build(2, 2, 600, 8, bias=7)
    r["bias_ids"][:, 6] = r["bias_ids"][:, 0]
    r["bias_ids"][:, 3] = r["bias_ids"][:, 2]
    check(z, r, torch.float32)


def test_counts_of_a_long_history_are_exact():
    z, r = build(1, 3, 100, 8, L=300000, bias=0, mask=False)
    r["history"][:] = 42
    r["draft"][:] = 42
    r["history_len"][:] = 300000
    r["prompt_len"][:] = 0
    check(z, r, torch.float32)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("V", [2048, 2051])
def test_addresses_that_are_not_aligned(dtype, V):
    """logits and out that begin on any element, alike or not."""
    z, r = build(2, 5, V, 21)
    z = z.to(dtype)
    want = call(z.cuda(), r)
    n = z.numel()
    for i, o in ((1, 0), (0, 1), (3, 3), (1, 2), (5, 5)):
        src = torch.zeros(n + 16, dtype=dtype, device="cuda")[i:i + n].view(z.shape)
        dst = torch.zeros(n + 16, dtype=dtype, device="cuda")[o:o + n].view(z.shape)
        src.copy_(z)
        assert torch.equal(call(src, r, out=dst), want)
        assert torch.equal(call(src, r, out=src), want)


def test_another_stream():
    z, r = build(4, 5, 32000, 2)
    want = call(z.cuda(), r)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    assert torch.equal(call(z.cuda(), r, stream=st), want)


def test_logits_beyond_32_bits():
    """Rows whose element offsets pass 2^31."""
    V, T, B = 152064, 17, 840  # 2.17e9 elements
    dev = torch.zeros((B, T, V), dtype=torch.bfloat16, device="cuda")
    z, r = build(2, T, V, 4, mask=False)
    dev[-2:] = z.to(torch.bfloat16).cuda()
    full = {k: np.concatenate([np.zeros((B - 2,) + x.shape[1:], x.dtype) if k != "repetition" else
                               np.ones((B - 2,), x.dtype), x]) for k, x in r.items()}
    full["bias_ids"][:-2] = -1
    got = call(dev, full, out=dev)[-2:].cpu().double().numpy()
    want, bound = R.logits(z.to(torch.bfloat16).float().numpy(), r, [T, T])
    assert (np.abs(got - want) <= bound + R.U_BF16 * np.abs(want)).all()
