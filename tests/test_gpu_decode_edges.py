"""The decode-step operators where their rules meet their limits: weights at a rounding boundary, sizes at which
another variant or another round of a loop begins, and calls that are captured or made on several streams."""
import pytest
import torch

import _decode as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


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
