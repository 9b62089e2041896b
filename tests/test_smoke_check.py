"""smoke()'s comparison of an operator's output with its definition (CPU only)."""
import math

import torch

from __graft_entry__ import agrees

F8, BF = torch.float8_e4m3fn, torch.bfloat16


def test_whole_numbers_are_exact():
    """Slots and positions, however large the others are."""
    want = torch.tensor([0, 3, 299, 1 << 20], dtype=torch.int32)
    assert agrees(want.clone(), want)
    for i in range(4):
        for off in (-1, 1, 2):
            got = want.clone()
            got[i] += off
            assert not agrees(got, want)


def test_what_is_moved_is_exact():
    want = torch.tensor([1e-6, 0.5, 3.0], dtype=torch.float64).float().double()
    assert agrees(want.float(), want, moved=True)
    assert not agrees(torch.nextafter(want.float(), torch.tensor(9.0)), want, moved=True)


def test_codes_are_within_half_a_step():
    x = torch.cat([torch.linspace(-448, 448, 9001, dtype=torch.float64), torch.linspace(-2.0 ** -5, 2.0 ** -5, 999, dtype=torch.float64)])
    code = x.float().to(F8)
    assert agrees(code, x)
    bits = code.view(torch.uint8).clone()
    bits[(bits & 0x7F) < 0x7D] += 2  # two steps off
    assert not agrees(bits.view(F8), x)
    one = code.view(torch.uint8).clone()
    one[-1] += 2
    assert not agrees(one.view(F8), x)


def test_others_go_by_their_type():
    want = torch.tensor([1.0, -100.0, -math.inf, 0.0], dtype=torch.float64)
    assert agrees(want.to(BF), want) and agrees(want.float(), want)
    assert not agrees((want + torch.tensor([1.0, 0, 0, 0])).to(BF), want)
    assert not agrees((want + torch.tensor([0.05, 0, 0, 0])).float(), want)
    assert agrees((want + torch.tensor([0.01, 0, 0, 0])).float(), want)
    assert not agrees(torch.tensor([1.0, -100.0, 0.0, 0.0]), want)
    assert not agrees(torch.tensor([math.nan, -100.0, -math.inf, 0.0]), want)
